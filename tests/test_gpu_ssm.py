"""GPU: the selective state space scan, its step and its backward against float64 (ssm_reference.py).

Tolerances count roundings.  bf16 rounds by at most 2^-8 of a value.  y: the result, and the terms'
operands (the state for C S, the decayed scores) once each: 2^-8 |y| + 2^-8 (1 + 2^-6) times the sum of
the terms' magnitudes.  dx and dB, dC the same with their operands.  States, ddt, dA, d(dt_bias) and
d(initial state) only see products whose operands are two or three bf16 parts (2^-16 of a term or less), FP32 sums and
decays whose exponents are FP32 sums: 2^-14 of the sum of magnitudes (two such factors and the
exponents); dD sums exact products in FP32: 2^-18 over these lengths.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import causal_depthwise_conv1d_width_amd as cc  # noqa: E402
import ssm_reference as ref  # noqa: E402

HALF, FINE = 2.0 ** -8 * (1 + 2.0 ** -6), 2.0 ** -14
TINY = 1e-30


def close(got, want, mag, own, terms, what):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    excess = (got - want).abs() - (own * want.abs() + terms * mag + TINY)
    at = int(excess.argmax()) if excess.numel() else 0
    assert excess.numel() == 0 or excess.max() <= 0, \
        f"{what}: off by {float((got - want).abs().flatten()[at]):.3g} at {at}, value {float(want.flatten()[at]):.3g}"


class Problem:
    def __init__(self, lens, H, P, G, N, *, seed=0, dt32=True, pad=0, wide=0, decay=4.0, step=-2.0, bounds=None):
        gen = torch.Generator().manual_seed(seed)

        def rnd(*shape, dtype=torch.bfloat16):
            return torch.randn(shape, generator=gen).to(dtype)

        R = sum(lens) + pad
        self.lens, self.R, self.dims = lens, R, (H, P, G, N)
        ends = torch.cumsum(torch.tensor(lens), 0).tolist()
        self.bounds = [(e - n, e) for n, e in zip(lens, ends)]
        self.cu = torch.tensor([0] + ends, dtype=torch.int32, device="cuda")
        row = rnd(R, H * P + 2 * G * N + wide).cuda()
        self.x = row[:, :H * P].view(R, H, P)
        self.B = row[:, H * P:H * P + G * N].view(R, G, N)
        self.C = row[:, H * P + G * N:H * P + 2 * G * N].view(R, G, N)
        self.dt = (0.7 * rnd(R, H, dtype=torch.float32)).to(torch.float32 if dt32 else torch.bfloat16).cuda()
        self.A = -(0.1 + decay * torch.rand(H, generator=gen)).cuda()
        self.D, self.bias = rnd(H, dtype=torch.float32).cuda(), (step + rnd(H, dtype=torch.float32)).cuda()
        n = len(lens)
        self.S0, self.dS = rnd(n, H, P, N, dtype=torch.float32).cuda(), rnd(n, H, P, N, dtype=torch.float32).cuda()
        self.dy = rnd(R, H, P).cuda()

    def args(self):
        return self.x, self.dt, self.A, self.B, self.C, self.D, self.bias

    def host(self):
        return [t.cpu() for t in self.args()]

    def reference(self, S0, **kw):
        out = []
        for m in (False, True):
            out.append(ref.scan(*self.host(), self.bounds, S0.cpu(), magnitudes=m, **kw))
        return out


def check_fwd(p, **kw):
    (y, fin, _), (ym, fm, _) = p.reference(p.S0)
    got_fin = torch.full_like(p.S0, float("nan"))
    got = cc.ssm_scan_fwd(*p.args(), initial_state=p.S0, final_state=got_fin, **(kw or dict(cu_seqlens=p.cu)))
    torch.cuda.synchronize()
    n = sum(p.lens)
    close(got[:n], y[:n], ym[:n], HALF, HALF, "y")
    close(got_fin, fin, fm, 0.0, FINE, "final_state")


def check_bwd(p, S0, dS, **kw):
    z = torch.zeros_like(p.S0)
    (_, _, g), (_, _, gm) = p.reference(z if S0 is None else S0, dy=p.dy.cpu(), dS=None if dS is None else dS.cpu())
    got = cc.ssm_scan_bwd(p.dy, *p.args(), initial_state=S0, dfinal_state=dS, **(kw or dict(cu_seqlens=p.cu)))
    torch.cuda.synchronize()
    n = sum(p.lens)
    out = HALF if p.dt.dtype == torch.bfloat16 else 0.0
    for k, own, terms in (("dx", HALF, HALF), ("dB", HALF, HALF), ("dC", HALF, HALF), ("ddt", out, FINE)):
        close(getattr(got, k)[:n], g[k][:n], gm[k][:n], own, terms, k)
    for k, terms in (("dA", FINE), ("ddt_bias", FINE), ("dD", 2.0 ** -18)):
        close(getattr(got, k), g[k], gm[k], 0.0, terms, k)
    if S0 is not None:
        close(got.dinitial_state, g["dS0"], gm["dS0"], 0.0, FINE, "dinitial_state")
    return got


SHAPES = [  # lens, H, P, G, N
    ([1], 1, 1, 1, 1),
    ([64], 2, 64, 1, 64),
    ([1, 0, 63, 65, 2, 0], 4, 64, 2, 128),
    ([130, 7], 3, 40, 3, 16),
    ([5, 200], 2, 128, 1, 72),
    ([77], 2, 72, 2, 200),
    ([70, 64, 1], 2, 13, 1, 37),
    ([100], 2, 64, 1, 256),
    ([0, 0, 3], 6, 32, 2, 129),
]


@pytest.mark.parametrize("lens,H,P,G,N", SHAPES)
@pytest.mark.parametrize("dt32", [True, False])
def test_scan_forward(lens, H, P, G, N, dt32):
    print(f"[gpu] scan fwd {lens} H={H} P={P} G={G} N={N} dt32={dt32}", flush=True)
    check_fwd(Problem(lens, H, P, G, N, dt32=dt32, pad=3, wide=5))


@pytest.mark.parametrize("lens,H,P,G,N", SHAPES)
@pytest.mark.parametrize("dt32", [True, False])
def test_scan_backward(lens, H, P, G, N, dt32):
    print(f"[gpu] scan bwd {lens} H={H} P={P} G={G} N={N} dt32={dt32}", flush=True)
    p = Problem(lens, H, P, G, N, dt32=dt32, pad=2, wide=3, seed=1)
    check_bwd(p, p.S0, p.dS)


def test_batch_rows_and_whole_array():
    p = Problem([96, 96, 96], 4, 64, 1, 64, seed=2)
    check_fwd(p, seqlen=96)
    check_bwd(p, None, None, seqlen=96)
    p = Problem([150], 4, 32, 2, 128, seed=3)
    y = cc.ssm_scan_fwd(*p.args())
    assert torch.equal(y, cc.ssm_scan_fwd(*p.args(), seqlen=150))


@pytest.mark.parametrize("lens", [[1500], [3, 1400, 40], [700, 701]])
def test_long_sequences_in_pieces(lens):
    """Few blocks of long sequences: pieces with a join."""
    print(f"[gpu] scan pieces {lens}", flush=True)
    p = Problem(lens, 2, 64, 1, 64, seed=4, step=-3.0)
    check_fwd(p)
    check_bwd(p, p.S0, p.dS)


@pytest.mark.parametrize("N", [40, 200])
def test_batch_rows_in_pieces(N):
    print(f"[gpu] scan batch rows in pieces N={N}", flush=True)
    p = Problem([1100, 1100], 2, 40, 1, N, seed=6, step=-3.0)
    check_fwd(p, seqlen=1100)
    check_bwd(p, None, None, seqlen=1100)


@pytest.mark.parametrize("decay,step", [(60.0, 2.0), (0.001, -6.0), (4.0, 25.0)])
def test_fast_and_slow_decay(decay, step):
    """Decays that leave nothing of a chunk's start, that keep everything, and softplus past its bend."""
    p = Problem([150, 20], 4, 64, 2, 64, seed=5, decay=decay, step=step)
    check_fwd(p)
    check_bwd(p, p.S0, p.dS)


def test_zero_steps_and_no_softplus():
    p = Problem([90], 4, 64, 2, 64, seed=6)
    p.dt = p.dt.abs()
    p.dt[5] = 0
    p.dt[64:70] = 0
    p.bias = torch.zeros_like(p.bias)
    (y, fin, _), (ym, fm, _) = p.reference(p.S0, sp=False)
    got_fin = torch.empty_like(p.S0)
    got = cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu, dt_softplus=False, initial_state=p.S0, final_state=got_fin)
    close(got, y, ym, HALF, HALF, "y")
    close(got_fin, fin, fm, 0.0, FINE, "final")
    (_, _, g), (_, _, gm) = p.reference(p.S0, sp=False, dy=p.dy.cpu(), dS=p.dS.cpu())
    b = cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, dt_softplus=False, initial_state=p.S0, dfinal_state=p.dS)
    close(b.ddt, g["ddt"], gm["ddt"], 0.0, FINE, "ddt")
    close(b.dx, g["dx"], gm["dx"], HALF, HALF, "dx")


def test_without_skip_and_bias():
    p = Problem([70, 9], 4, 64, 2, 64, seed=7)
    x, dt, A, B, C = p.args()[:5]
    p.D, p.bias = torch.zeros_like(p.D), torch.zeros_like(p.bias)
    assert torch.equal(cc.ssm_scan_fwd(x, dt, A, B, C, cu_seqlens=p.cu), cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu))
    got = cc.ssm_scan_bwd(p.dy, x, dt, A, B, C, cu_seqlens=p.cu)
    full = cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu)
    assert got.dD is None and got.ddt_bias is None and got.dinitial_state is None
    for k in ("dx", "ddt", "dA", "dB", "dC"):
        assert torch.equal(getattr(got, k), getattr(full, k)), k


def test_pool_slots():
    """Slots, a -1, an out-of-range slot, unread start states, an empty sequence, and untouched rows."""
    H, P, G, N = 4, 64, 2, 72
    p = Problem([70, 0, 5, 33, 130], H, P, G, N, seed=8, pad=4)
    pool = torch.randn(8, H, P, N, device="cuda") * 0.5
    before = pool.clone()
    ci = torch.tensor([6, 2, -1, 9, 0], dtype=torch.int32, device="cuda")
    hi = torch.tensor([1, 1, 1, 1, 0], dtype=torch.uint8, device="cuda")
    out = torch.full((p.R, H, P), 7.0, dtype=torch.bfloat16, device="cuda")
    cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu, state_pool=pool, cache_indices=ci, has_initial_state=hi, out=out)
    S0 = torch.zeros(5, H, P, N)
    S0[0] = before[6].cpu()
    (y, fin, _), (ym, fm, _) = p.reference(S0)
    for i in (0, 4):
        s, e = p.bounds[i]
        close(out[s:e], y[s:e], ym[s:e], HALF, HALF, f"y of sequence {i}")
        close(pool[int(ci[i])], fin[i], fm[i], 0.0, FINE, f"state of sequence {i}")
    for i in (2, 3):
        s, e = p.bounds[i]
        assert (out[s:e].view(torch.int16) == 0).all()
    assert (out[sum(p.lens):] == 7).all()
    for slot in (1, 2, 3, 4, 5, 7):
        assert torch.equal(pool[slot], before[slot])
    # no flags: all start from zeros
    pool2 = before.clone()
    cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu, state_pool=pool2, cache_indices=ci)
    (_, fin, _), (_, fm, _) = p.reference(torch.zeros_like(S0))
    close(pool2[6], fin[0], fm[0], 0.0, FINE, "state without flags")
    assert torch.equal(pool2[2], before[2])


def test_pool_with_wide_slots():
    p = Problem([40, 41], 2, 64, 1, 64, seed=9)
    big = torch.randn(4, 3, 64, 64, device="cuda")
    pool, keep = big[:, :2], big[:, 2].clone()
    ci = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    S0 = pool[ci.long()].clone()
    cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu, state_pool=pool, cache_indices=ci,
                    has_initial_state=torch.ones(2, dtype=torch.bool, device="cuda"))
    (_, fin, _), (_, fm, _) = p.reference(S0)
    close(pool[ci.long()], fin, fm, 0.0, FINE, "pool")
    assert torch.equal(big[:, 2], keep)


@pytest.mark.parametrize("H,P,G,N", [(1, 1, 1, 1), (4, 64, 2, 128), (3, 20, 3, 16), (2, 130, 1, 30), (2, 64, 1, 63),
                                     (4, 48, 1, 256), (6, 9, 2, 12)])
@pytest.mark.parametrize("n", [1, 7])
def test_state_update(H, P, G, N, n):
    print(f"[gpu] step n={n} H={H} P={P} G={G} N={N}", flush=True)
    p = Problem([1] * n, H, P, G, N, seed=10, wide=3, dt32=n == 1)
    pool = torch.randn(n + 3, H, P, N, device="cuda")
    before = pool.clone()
    ci = torch.randperm(n + 3)[:n].to(torch.int32).cuda()
    if n > 1:
        ci[3] = -1
    got = cc.ssm_state_update(*p.args(), state_pool=pool, cache_indices=ci)
    S0 = before[ci.long()].clone()
    (y, fin, _), (ym, fm, _) = p.reference(S0)
    live = [i for i in range(n) if int(ci[i]) >= 0]
    # FP32 throughout: y is rounded once, sums of N terms
    close(got[live], y[live], ym[live], HALF, 2.0 ** -18, "y")
    close(pool[ci[live].long()], fin[live], fm[live], 0.0, 2.0 ** -20, "state")
    if n > 1:
        assert (got[3].view(torch.int16) == 0).all()
    rest = sorted(set(range(n + 3)) - set(ci.tolist()))
    assert torch.equal(pool[rest], before[rest])


def test_steps_follow_a_prompt():
    """A prompt in one call, in two calls through the pool, and its last rows as single steps."""
    H, P, G, N = 4, 64, 2, 64
    p = Problem([100], H, P, G, N, seed=11)
    pool = torch.zeros(3, H, P, N, device="cuda")
    ci = torch.tensor([1], dtype=torch.int32, device="cuda")
    on = torch.ones(1, dtype=torch.uint8, device="cuda")
    x, dt, A, B, C, D, b = p.args()
    cc.ssm_scan_fwd(x[:60], dt[:60], A, B[:60], C[:60], D, b, state_pool=pool, cache_indices=ci)
    cc.ssm_scan_fwd(x[60:95], dt[60:95], A, B[60:95], C[60:95], D, b, state_pool=pool, cache_indices=ci, has_initial_state=on)
    (y, fin, _), (ym, fm, _) = p.reference(torch.zeros(1, H, P, N))
    for t in range(95, 100):
        r = slice(t, t + 1)
        yt = cc.ssm_state_update(x[r], dt[r], A, B[r], C[r], D, b, state_pool=pool, cache_indices=ci)
        close(yt, y[r], ym[r], HALF, HALF, f"y of row {t}")
    close(pool[1:2], fin, fm, 0.0, FINE, "state")


def test_same_bits_and_other_streams():
    p = Problem([300, 77, 5], 4, 64, 2, 128, seed=12, dt32=False)
    y0 = cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu)
    g0 = cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, initial_state=p.S0, dfinal_state=p.dS)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        ws = torch.randint(0, 255, (cc.ssm_scan_bwd_workspace_bytes(p.x, p.dt, p.B, 3) + 64,), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        y = cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu, stream=stream)
        g = cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, initial_state=p.S0, dfinal_state=p.dS, workspace=ws[16:], stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(y, y0)
        for a, b in zip(g, g0):
            assert torch.equal(a, b)


def test_graph_replays():
    p = Problem([200, 56], 4, 64, 2, 64, seed=13)
    pool = torch.randn(3, *p.S0.shape[1:], device="cuda")
    ci = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    on = torch.ones(2, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def work():
        y = cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu, state_pool=pool, cache_indices=ci, has_initial_state=on)
        g = cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, initial_state=p.S0)
        s = cc.ssm_state_update(p.x[:2], p.dt[:2], p.A, p.B[:2], p.C[:2], p.D, p.bias, state_pool=pool, cache_indices=ci)
        return [y, s, *[t for t in g if t is not None]]

    start = pool.clone()
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for k in range(3):
        p.x.mul_(0.5)
        pool.copy_(start)
        want = [t.clone() for t in work()]
        end = pool.clone()
        pool.copy_(start)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool, end), k
        for a, b in zip(captured, want):
            assert torch.equal(a, b), k


def test_gradient_into_wider_rows():
    """dx, dB, dC as column ranges of one array, as the convolution's backward takes them."""
    H, P, G, N = 4, 64, 2, 64
    p = Problem([150, 31], H, P, G, N, seed=14)
    want = cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu)
    row = torch.full((p.R, H * P + 2 * G * N + 6), 3.0, dtype=torch.bfloat16, device="cuda")
    dx = row[:, 2:2 + H * P].view(p.R, H, P)
    dB = row[:, 2 + H * P:2 + H * P + G * N].view(p.R, G, N)
    dC = row[:, 2 + H * P + G * N:2 + H * P + 2 * G * N].view(p.R, G, N)
    got = cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, dx=dx, dB=dB, dC=dC)
    for k in ("dx", "dB", "dC", "ddt", "dA"):
        assert torch.equal(getattr(got, k), getattr(want, k)), k
    assert (row[:, :2] == 3).all() and (row[:, -4:] == 3).all()


def test_gradient_against_differences():
    """The final state is FP32: its change along directions of dt and A against the gradients."""
    p = Problem([90, 40], 2, 64, 1, 64, seed=15, step=-1.5)
    zero = torch.zeros_like(p.dy)
    g = cc.ssm_scan_bwd(zero, *p.args(), cu_seqlens=p.cu, initial_state=p.S0, dfinal_state=p.dS)

    def loss(dt, A):
        fin = torch.empty_like(p.S0)
        cc.ssm_scan_fwd(p.x, dt, A, p.B, p.C, p.D, p.bias, cu_seqlens=p.cu, initial_state=p.S0, final_state=fin)
        return (fin.double() * p.dS.double()).sum()

    gen = torch.Generator().manual_seed(1)
    v = torch.randn(p.dt.shape, generator=gen).cuda()
    vA = torch.randn(p.A.shape, generator=gen).cuda()
    for eps, f, want in ((2.0 ** -7, lambda e: loss(p.dt + e * v, p.A), (g.ddt.double() * v).sum()),
                         (2.0 ** -7, lambda e: loss(p.dt, p.A + e * vA), (g.dA.double() * vA).sum())):
        slope = (f(eps) - f(-eps)) / (2 * eps)
        half = (f(eps / 2) - f(-eps / 2)) / eps
        slope = (4 * half - slope) / 3  # fourth order in eps
        scale = (p.dS.double().abs().sum() * 4) * 2.0 ** -14 / eps  # states are right to 2^-14 of their terms
        assert abs(float(slope - want)) <= float(1e-3 * want.abs() + scale * 2.0 ** -5), (float(slope), float(want))


def test_offsets_past_32_bits():
    """A row stride that puts the last rows past 2^31 elements; pool slots likewise."""
    H, P, G, N = 2, 64, 1, 64
    p = Problem([140], H, P, G, N, seed=16)
    ld = 1 << 24
    wide = torch.empty((140 * ld,), dtype=torch.bfloat16, device="cuda").view(140, ld)
    x = wide[:, 8:8 + H * P].view(140, H, P)
    x.copy_(p.x)
    assert torch.equal(cc.ssm_scan_fwd(x, *p.args()[1:]), cc.ssm_scan_fwd(*p.args()))
    a = cc.ssm_scan_bwd(p.dy, x, *p.args()[1:])
    for u, v in zip(a, cc.ssm_scan_bwd(p.dy, *p.args())):
        assert u is None and v is None or torch.equal(u, v)
    del wide, x
    pool = torch.empty((3, (1 << 30)), dtype=torch.float32, device="cuda")[:, :H * P * N].view(3, H, P, N)
    pool.copy_(torch.randn(3, H, P, N, device="cuda"))
    small = pool.clone()
    ci = torch.tensor([2], dtype=torch.int32, device="cuda")
    for t in (pool, small):
        cc.ssm_scan_fwd(*p.args(), state_pool=t, cache_indices=ci, has_initial_state=torch.ones(1, dtype=torch.uint8, device="cuda"))
        cc.ssm_state_update(p.x[:1], p.dt[:1], p.A, p.B[:1], p.C[:1], p.D, p.bias, state_pool=t, cache_indices=ci)
    assert torch.equal(pool, small)


def test_no_rows():
    H, P, G, N = 2, 64, 1, 64
    p = Problem([0, 0], H, P, G, N, seed=17)
    fin = torch.full_like(p.S0, float("nan"))
    assert cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu, initial_state=p.S0, final_state=fin).shape == (0, H, P)
    assert torch.equal(fin, p.S0)
    g = cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, initial_state=p.S0, dfinal_state=p.dS)
    assert torch.equal(g.dinitial_state, p.dS)
    assert not g.dA.any() and not g.dD.any() and not g.ddt_bias.any()
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=none)
    assert not g.dA.any()
