"""GPU: the gated delta rule and its step against float64 (delta_reference.py).

Tolerances count roundings.  bf16 rounds by at most 2^-8 of a value.  y: the result, and each term's operand (the state
or the decayed score) once: 2^-8 |y| + 2^-8 (1 + 2^-6) times the sum of the terms' magnitudes (for operands of one bf16
part; the kernels' have 2^-12 and 2^-17).  A state's rounding errors
are those of FP32 sums: in a chunk at most 40 roundings (12 accumulations of K S, 12 of T R, 6 of K^T U, decays and
splits) of 2^-24 of a column's largest sum of magnitudes, over at most 8 chunks, none grown by a later chunk (decays and
I - r k k^T have norms of at most one for |k|^2 r <= 2): 8 * 40 * 2^-24 < 2^-15.  The step is FP32 throughout: sums of 256
terms in four by shuffles, at most 16 roundings, twice: 2^-18 of the magnitudes, and the result's bf16 rounding.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import causal_depthwise_conv1d_width_amd as cc  # noqa: E402
import delta_reference as ref  # noqa: E402

bf16, f32 = torch.bfloat16, torch.float32
HALF, FINE, TINY = 2.0 ** -8 * (1 + 2.0 ** -6), 2.0 ** -15, 1e-30


def within(got, want, allowed, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    excess = (got - want).abs() - allowed - TINY
    at = int(excess.argmax()) if excess.numel() else 0
    assert excess.numel() == 0 or excess.max() <= 0, \
        f"{what}: off by {float((got - want).abs().flatten()[at]):.3g} at {at}, value {float(want.flatten()[at]):.3g}"


class Problem:
    """q, k, v are column ranges of one row array; `pad` rows behind the last sequence belong to none."""

    def __init__(self, lens, H, P, G, N, *, seed=0, gates=f32, norm=True, beta=1.0, pad=0, wide=0, decay=4.0, key=1.0,
                 first=0, **kw):
        gen = torch.Generator().manual_seed(seed)

        def rnd(*shape, dtype=bf16):
            return torch.randn(shape, generator=gen).to(dtype)

        R = first + sum(lens) + pad
        self.lens, self.R, self.dims = lens, R, (H, P, G, N)
        ends = [first + int(e) for e in torch.cumsum(torch.tensor(lens), 0)]
        self.bounds = [(e - n, e) for n, e in zip(lens, ends)]
        self.cu = torch.tensor([first] + ends, dtype=torch.int32, device="cuda")
        row = rnd(R, H * P + 2 * G * N + wide)
        row[:, G * N:2 * G * N] = row[:, G * N:2 * G * N] * (key if norm else key * N ** -0.5) + (0.5 * key if norm else 0)
        row = row.cuda()
        self.q = row[:, :G * N].view(R, G, N)
        self.k = row[:, G * N:2 * G * N].view(R, G, N)
        self.v = row[:, 2 * G * N:2 * G * N + H * P].view(R, H, P)
        self.dt, self.b = (0.7 * rnd(R, H, dtype=f32)).to(gates).cuda(), rnd(R, H, dtype=f32).to(gates).cuda()
        self.A = -(0.1 + decay * torch.rand(H, generator=gen)).cuda()
        self.bias = (rnd(H, dtype=f32) - 2.0).cuda()
        n = len(lens)
        self.S0, self.dS = rnd(n, H, P, N, dtype=f32).cuda(), rnd(n, H, P, N, dtype=f32).cuda()
        self.dy = rnd(R, H, P).cuda()
        self.kw = dict(qk_norm=norm, beta_max=beta, **kw)

    def args(self):
        return self.q, self.k, self.v, self.dt, self.b, self.A, self.bias

    def reference(self, S0=None, bounds=None, args=None):
        n = {"qk_norm": "norm", "beta_max": "beta", "norm_eps": "eps", "dt_softplus": "softplus", "scale": "scale"}
        H, P, _, N = self.dims
        zero = torch.zeros(len(self.lens), H, P, N)
        return ref.rule(*((t.cpu() if t is not None else None) for t in (args or self.args())), bounds or self.bounds,
                        zero if S0 is None else S0.cpu(), **{n[m]: x for m, x in self.kw.items()})

    def check(self, y, final, want, what=""):
        wy, wf, (my, mf) = want
        rows = [t for s, e in self.bounds for t in range(s, e)]
        within(y[rows], wy[rows], 2.0 ** -8 * wy[rows].abs() + HALF * my[rows], what + "y")
        if final is not None:
            within(final, wf, FINE * mf.amax(-1, keepdim=True), what + "states")


SHAPES = [  # lens, H, P, G, N
    ([130], 2, 64, 1, 64), ([1], 1, 16, 1, 16), ([64, 64], 4, 128, 2, 128), ([63, 0, 65, 1], 3, 64, 1, 128),
    ([200, 37], 2, 40, 2, 72), ([100], 2, 33, 1, 37), ([70, 5], 2, 130, 1, 200), ([300], 1, 64, 1, 256), ([9], 2, 8, 2, 1),
    ([450], 2, 64, 2, 32)]


@pytest.mark.parametrize("lens,H,P,G,N", SHAPES, ids=str)
@pytest.mark.parametrize("kind", ["norm", "raw"])
def test_forward(lens, H, P, G, N, kind):
    p = Problem(lens, H, P, G, N, seed=len(lens) + N, norm=kind == "norm", beta=1.0 if kind == "norm" else 1.5,
                gates=f32 if kind == "norm" else bf16, wide=5 if kind == "raw" else 0, key=0.8 if kind == "raw" else 1.0)
    final = torch.full((len(lens), H, P, N), float("nan"), device="cuda")
    y = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, initial_state=p.S0, final_state=final, **p.kw)
    p.check(y, final, p.reference(p.S0))
    y0 = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, **p.kw)
    p.check(y0, None, p.reference())


def test_batch_rows_and_default_sequence():
    p = Problem([75, 75], 2, 64, 2, 64, seed=5)
    a = cc.delta_scan_fwd(*p.args(), seqlen=75, **p.kw)
    b = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, **p.kw)
    assert torch.equal(a, b)
    one = Problem([150], 2, 64, 2, 64, seed=5)
    one.check(cc.delta_scan_fwd(*one.args(), **one.kw), None, one.reference())


@pytest.mark.parametrize("kw", [dict(scale=1.0), dict(dt_softplus=False), dict(norm_eps=0.1), dict(beta=2.0)], ids=str)
def test_options(kw):
    p = Problem([90, 20], 2, 32, 1, 48, seed=3, **kw)
    if "dt_softplus" in kw:
        p.dt = p.dt.abs() * 0.2
        p.bias = p.bias.abs() * 0.1
    final = torch.empty(2, 2, 32, 48, device="cuda")
    y = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, final_state=final, **p.kw)
    p.check(y, final, p.reference())
    args = (*p.args()[:6], None)
    y = cc.delta_scan_fwd(*args, cu_seqlens=p.cu, final_state=final, **p.kw)
    p.check(y, final, p.reference(args=args), "no bias: ")


def test_correlated_keys():
    """Keys that are almost one direction, little decay and rates near two: the triangular system is far from the identity."""
    p = Problem([128], 2, 64, 1, 64, seed=9, beta=2.0, decay=0.01, key=0.05)
    p.k.add_(1.0)
    p.b.add_(3.0)
    final = torch.empty(1, 2, 64, 64, device="cuda")
    y = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, final_state=final, **p.kw)
    p.check(y, final, p.reference())


def test_pool():
    """Slots in any order, one absent, flags; untouched slots and rows outside the sequences keep their bits."""
    p = Problem([70, 0, 65, 20, 33], 2, 40, 1, 64, seed=11, pad=7, first=3)
    H, P, G, N = p.dims
    wide = torch.randn(9, H * P * N + 8, device="cuda")
    pool = wide[:, :H * P * N].view(9, H, P, N)
    ci = torch.tensor([4, 2, 7, -1, 0], dtype=torch.int32, device="cuda")
    hi = torch.tensor([1, 1, 0, 1, 1], dtype=torch.uint8, device="cuda")
    before = wide.clone()
    out = torch.full((p.R, H, P), 3.0, dtype=bf16, device="cuda")
    y = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, state_pool=pool, cache_indices=ci, has_initial_state=hi, out=out, **p.kw)
    S0 = before[:, :H * P * N].view(9, H, P, N)[ci.clamp(min=0).long()] * hi[:, None, None, None]
    wy, wf, (my, mf) = p.reference(S0)
    s, e = p.bounds[3]
    wy[s:e], my[s:e] = 0, 0
    live = [0, 2, 4]
    p.check(y, None, (wy, None, (my, None)))
    assert (y[s:e].view(torch.int16) == 0).all()
    within(pool[ci.long()[live]], wf[live], FINE * mf[live].amax(-1, keepdim=True), "pool")
    same = [i for i in range(9) if i not in (4, 7, 0)]
    assert torch.equal(wide[same], before[same]) and torch.equal(wide[:, H * P * N:], before[:, H * P * N:])
    assert (y[:3] == 3.0).all() and (y[-7:] == 3.0).all()
    pool2 = before[:, :H * P * N].reshape(9, H, P, N).contiguous()
    cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, state_pool=pool2, cache_indices=ci, **p.kw)  # no flags: from zeros
    within(pool2[ci.long()[live]], p.reference()[1][live], FINE * mf[live].amax(-1, keepdim=True), "pool from zeros")


def test_empty_sequences_pass_states_on():
    p = Problem([0, 5, 0], 2, 16, 1, 16, seed=2)
    final = torch.full((3, 2, 16, 16), float("nan"), device="cuda")
    cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, initial_state=p.S0, final_state=final, **p.kw)
    assert torch.equal(final[0], p.S0[0]) and torch.equal(final[2], p.S0[2])
    none = Problem([0, 0], 2, 16, 1, 16, seed=2)
    final = torch.full((2, 2, 16, 16), float("nan"), device="cuda")
    y = cc.delta_scan_fwd(*none.args(), cu_seqlens=none.cu, initial_state=none.S0, final_state=final, **none.kw)
    assert y.shape == (0, 2, 16) and torch.equal(final, none.S0)


def test_step_follows_prefill():
    """A prompt in one call, and the same prompt as a prefill of its first rows and then token by token."""
    p = Problem([40, 40], 4, 33, 2, 50, seed=21, beta=1.7)
    H, P, G, N = p.dims
    pool = torch.zeros(3, H, P, N, device="cuda")
    ci = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    want = p.reference()
    rows = [torch.arange(s, s + 30) for s, _ in p.bounds]
    first = torch.cat(rows).cuda()
    part = tuple(t[first] for t in p.args()[:5])
    cc.delta_scan_fwd(*part, p.A, p.bias, seqlen=30, state_pool=pool, cache_indices=ci, **p.kw)
    for j in range(30, 40):
        at = torch.tensor([s + j for s, _ in p.bounds]).cuda()
        y = cc.delta_state_update(*(t[at] for t in p.args()[:5]), p.A, p.bias, state_pool=pool, cache_indices=ci, **p.kw)
        wy, my = want[0][at.cpu()], want[2][0][at.cpu()]
        within(y, wy, 2.0 ** -8 * wy.abs() + FINE * my, f"token {j}")
    within(pool[ci.long()], want[1], FINE * want[2][1].amax(-1, keepdim=True), "states")
    assert (pool[1] == 0).all()


@pytest.mark.parametrize("n,H,P,G,N", [(1, 1, 16, 1, 16), (5, 4, 64, 2, 128), (3, 3, 52, 1, 100), (2, 2, 7, 1, 37),
                                       (4, 2, 130, 2, 256), (2, 1, 3, 1, 1), (3, 2, 64, 1, 20)], ids=str)
@pytest.mark.parametrize("kind", ["norm", "raw"])
def test_step(n, H, P, G, N, kind):
    p = Problem([1] * n, H, P, G, N, seed=N, norm=kind == "norm", gates=bf16 if kind == "norm" else f32, wide=3, beta=1.5)
    pool = torch.randn(n + 3, H, P, N, device="cuda")
    before = pool.clone()
    ci = torch.arange(n, dtype=torch.int32).flip(0).cuda() + 1
    y = cc.delta_state_update(*p.args(), state_pool=pool, cache_indices=ci, **p.kw)
    wy, wf, (my, mf) = p.reference(before[ci.long()])
    within(y, wy, 2.0 ** -8 * wy.abs() + 2.0 ** -18 * my, "y")
    within(pool[ci.long()], wf, 2.0 ** -18 * mf.amax(-1, keepdim=True), "states")
    assert torch.equal(pool[[0, n + 1, n + 2]], before[[0, n + 1, n + 2]])
    ci[0] = -1
    if n > 1:
        ci[1] = n + 3  # outside the pool: as -1
    before = pool.clone()
    y = cc.delta_state_update(*p.args(), state_pool=pool, cache_indices=ci, **p.kw)
    assert (y[:2].view(torch.int16) == 0).all()
    gone = [n, n - 1] if n > 1 else [n]
    assert torch.equal(pool[gone], before[gone])


@pytest.mark.parametrize("row", [0, 17, 63, 64, 99])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["v", "k", "dt", "b", "q"])
def test_not_finite_stays(row, value, where):
    """Rows before, other sequences, other heads, and, for v, other columns keep their bits."""
    p = Problem([100, 30], 4, 20, 2, 40, seed=13)
    final = torch.empty(2, 4, 20, 40, device="cuda")
    clean = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, final_state=final, **p.kw)
    f_clean = final.clone()
    t = dict(v=p.v, k=p.k, q=p.q, dt=p.dt, b=p.b)[where]
    if where == "b" and value > 0:
        value = float("nan")  # a rate of an infinite b is finite
    if where == "dt" and value > 0:
        value = float("nan")  # an infinite step is a decay to zero
    if t.dim() == 3:
        t[row, 1, 3] = value
    else:
        t[row, 1] = value
    y = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, final_state=final, **p.kw)
    hit = torch.zeros_like(y, dtype=torch.bool)
    if where == "v":
        hit[row:100, 1, 3] = True
    elif where == "k":
        hit[row:100, 2:4] = True
    elif where == "q":
        hit[row, 2:4] = True
    else:
        hit[row:100, 1] = True
    assert torch.equal(y[~hit], clean[~hit])
    assert not torch.isfinite(y[hit]).any()
    keep = torch.ones_like(final, dtype=torch.bool)
    if where == "v":
        keep[0, 1, 3] = False
    elif where == "k":
        keep[0, 2:4] = False
    elif where != "q":
        keep[0, 1] = False
    assert torch.equal(final[keep], f_clean[keep])
    assert not torch.isfinite(final[~keep]).any()


def test_infinite_gates():
    """b = -inf: no write; dt = inf: the state is forgotten; both are finite."""
    p = Problem([100], 2, 16, 1, 32, seed=17)
    p.b[10:30] = -float("inf")
    p.b[70] = float("inf")
    p.dt[50] = float("inf")
    final = torch.empty(1, 2, 16, 32, device="cuda")
    y = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, initial_state=p.S0, final_state=final, **p.kw)
    p.dt[50] = 1e4  # a step as good as infinite, that the reference can take
    p.check(y, final, p.reference(p.S0))


def test_rows_of_no_sequence_hold_anything():
    p = Problem([50, 40], 2, 24, 1, 32, seed=19, pad=9, first=5)
    want = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, **p.kw)
    for t in (p.q, p.k, p.v, p.dt, p.b):
        t[:5] = float("nan")
        t[-9:] = float("inf")
    got = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, **p.kw)
    assert torch.equal(got[5:-9], want[5:-9])


def test_same_bits_any_workspace_and_stream():
    p = Problem([90, 70, 200], 4, 64, 2, 128, seed=23)
    final = torch.empty(3, 4, 64, 128, device="cuda")
    y = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, final_state=final, **p.kw)
    need = cc.delta_scan_fwd_workspace_bytes(p.v, p.k, p.dt, 3)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device="cuda")
    f2 = torch.empty_like(final)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2 = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, final_state=f2, workspace=ws[16:16 + need], stream=s, **p.kw)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, y2) and torch.equal(final, f2)
    assert (ws[:16] == 0xff).all() and (ws[16 + need:] == 0xff).all()


def test_captured_prefill_and_decode():
    """A prefill and three steps in one graph, replayed with new inputs between eager work."""
    p = Problem([60, 50], 2, 32, 1, 64, seed=29)
    H, P, G, N = p.dims
    pool = torch.zeros(4, H, P, N, device="cuda")
    ci = torch.tensor([3, 1], dtype=torch.int32, device="cuda")

    def work():
        y = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, state_pool=pool, cache_indices=ci, **p.kw)
        ys = [y]
        for j in range(3):
            ys.append(cc.delta_state_update(*(t[j:j + 2] for t in p.args()[:5]), p.A, p.bias, state_pool=pool,
                                            cache_indices=ci, **p.kw))
        return ys

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for k in range(3):
        p.v.mul_(-0.5)
        p.k.add_(0.25)
        graph.replay()
        torch.cuda.synchronize()
        got, state = [t.clone() for t in captured], pool.clone()
        pool.zero_()
        want = work()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(state, pool)
        torch.randn(1000, device="cuda").sum().item()


def test_large_offsets():
    """Rows and slots whose offsets pass 32 bits."""
    H, P, G, N = 2, 16, 1, 16
    wide = 1 << 22
    R = 600
    p = Problem([R], H, P, G, N, seed=31)
    big = torch.empty(R, wide, dtype=bf16, device="cuda")
    big[:, -H * P:] = p.v.reshape(R, -1)
    v = big[:, -H * P:].unflatten(1, (H, P))
    slots = torch.empty(5, 1 << 29, device="cuda")
    pool = slots[:, :H * P * N].view(5, H, P, N)
    pool.copy_(torch.randn(5, H, P, N))
    start = pool[4].clone()
    ci = torch.tensor([4], dtype=torch.int32, device="cuda")
    hi = torch.ones(1, dtype=torch.uint8, device="cuda")
    y = cc.delta_scan_fwd(p.q, p.k, v, p.dt, p.b, p.A, p.bias, cu_seqlens=p.cu, state_pool=pool, cache_indices=ci,
                          has_initial_state=hi, **p.kw)
    final = torch.empty(1, H, P, N, device="cuda")
    y2 = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, initial_state=start[None], final_state=final, **p.kw)
    assert torch.equal(y, y2) and torch.equal(pool[4], final[0])
