"""GPU: the scan where it went wrong once: bits of calls in many pieces, calls on a stream of their own,
rows outside every sequence, NaN steps,
slow decays after sudden ones, values that are not finite.

Tolerances are those of test_gpu_ssm.py, whose problems and checks are used."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import causal_depthwise_conv1d_width_amd as cc  # noqa: E402
import test_gpu_ssm as base  # noqa: E402


@pytest.mark.parametrize("lens", [[1500], [2100, 3, 1300]])
def test_backward_in_many_pieces_has_the_same_bits(lens):
    """Pieces between a sequence's first and last are walked in both directions at once."""
    print(f"[gpu] bits of {lens}", flush=True)
    p = base.Problem(lens, 4, 64, 2, 64, seed=20, step=-3.0)
    need = cc.ssm_scan_bwd_workspace_bytes(p.x, p.dt, p.B, len(lens))
    want = base.check_bwd(p, p.S0, p.dS)
    for k in range(6):
        ws = torch.full((need + 4096 * k,), 255 * (k % 2), dtype=torch.uint8, device="cuda")  # zeros or NaN
        got = cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, initial_state=p.S0, dfinal_state=p.dS, workspace=ws)
        for name, a, b in zip(want._fields, got, want):
            assert torch.equal(a, b), (k, name)


def busy():
    """Work ahead of everything that the current stream gets from here on."""
    torch.cuda._sleep(200_000_000)


def test_pool_without_flags_on_another_stream():
    """The prompts start from zeros although the current stream is busy and the slots hold values."""
    p = base.Problem([200, 70], 4, 64, 2, 64, seed=21)
    before = torch.randn(4, 4, 64, 64, device="cuda")
    ci = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pools = [before.clone() for _ in range(2)]
    # memory that a small array on the current stream would get: bytes that are not zero
    stale = [torch.full((2,), 1, dtype=torch.uint8, device="cuda") for _ in range(8)]
    out, side = torch.empty_like(p.x, memory_format=torch.contiguous_format), torch.cuda.Stream()
    torch.cuda.synchronize()
    del stale
    busy()
    cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu, state_pool=pools[0], cache_indices=ci, out=out, stream=side)
    torch.cuda.synchronize()
    want = cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu, state_pool=pools[1], cache_indices=ci,
                           has_initial_state=torch.zeros(2, dtype=torch.uint8, device="cuda"))
    assert torch.equal(out, want) and torch.equal(pools[0], pools[1])
    assert torch.equal(pools[0][[0, 2]], before[[0, 2]]) and not torch.equal(pools[0][1], before[1])


def test_work_arrays_of_another_stream():
    """Calls on a side stream while the current stream still writes memory that it has given back."""
    p = base.Problem([1300, 40], 4, 64, 2, 64, seed=22, step=-3.0)
    m = torch.randn(300, 256, device="cuda").bfloat16()
    w, side = torch.rand(256, device="cuda"), torch.cuda.Stream()

    def work(**k):
        fin = torch.empty_like(p.S0) if not k else keep
        y = cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu, initial_state=p.S0, final_state=fin, **k)
        g = cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, initial_state=p.S0, dfinal_state=p.dS, **k)
        return [y, fin, *g, *cc.gated_norm_bwd(m, m, m, w, **k), *cc.residual_norm_bwd(m, m, m, w, **k)]

    want = work()
    need = cc.ssm_scan_bwd_workspace_bytes(p.x, p.dt, p.B, 2)
    keep = torch.empty_like(p.S0)
    torch.cuda.synchronize()
    busy()
    for size in (need, 1 << 20, 1 << 16, 1 << 10):
        for _ in range(6):
            torch.empty((size,), dtype=torch.uint8, device="cuda").fill_(255)  # NaN, written when the sleep ends
    got = work(stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_rows_before_the_first_sequence():
    """Offsets that begin past row 0: the rows before them belong to no sequence, like those after the last."""
    H, P, G, N = 4, 64, 1, 64
    p = base.Problem([9, 100, 30], H, P, G, N, seed=23, pad=4)
    cu, S0, dS = p.cu[1:].contiguous(), p.S0[1:].contiguous(), p.dS[1:].contiguous()
    bounds, (s, e) = p.bounds[1:], (9, 139)
    (y, _, g), (ym, _, gm) = [base.ref.scan(*p.host(), bounds, S0.cpu(), dy=p.dy.cpu(), dS=dS.cpu(), magnitudes=m)
                              for m in (False, True)]
    new = {k: torch.full_like(t, 7.0, memory_format=torch.contiguous_format)
           for k, t in dict(dx=p.x, ddt=p.dt, dB=p.B, dC=p.C).items()}
    ws = torch.full((cc.ssm_scan_bwd_workspace_bytes(p.x, p.dt, p.B, 2),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((p.R, H, P), 7.0, dtype=torch.bfloat16, device="cuda")
    cc.ssm_scan_fwd(*p.args(), cu_seqlens=cu, initial_state=S0, out=out)
    got = cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=cu, initial_state=S0, dfinal_state=dS, workspace=ws, **new)
    base.close(out[s:e], y[s:e], ym[s:e], base.HALF, base.HALF, "y")
    for k, own, terms in (("dx", base.HALF, base.HALF), ("dB", base.HALF, base.HALF), ("dC", base.HALF, base.HALF),
                          ("ddt", 0.0, base.FINE)):
        base.close(getattr(got, k)[s:e], g[k][s:e], gm[k][s:e], own, terms, k)
    for k, t in dict(new, y=out).items():
        assert (t[:s] == 7).all() and (t[e:] == 7).all(), k


def same_but(got, want, at, what):
    """got has want's bits outside `at`."""
    a, b = got.clone(), want.clone()
    a[at] = b[at] = 0
    assert torch.equal(a, b), what


@pytest.mark.parametrize("dt32", [True, False])
def test_nan_step_is_seen(dt32):
    """A NaN step makes its head NaN from its row on, and nothing else; -inf is a step of zero."""
    H, P, G, N, h, t = 4, 64, 2, 64, 2, 90
    p = base.Problem([50, 70, 30], H, P, G, N, seed=24, dt32=dt32)
    rows = slice(t, 120)  # the second sequence's from row t on

    def run():
        fin = torch.empty_like(p.S0)
        y = cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu, initial_state=p.S0, final_state=fin)
        return y, fin, cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, initial_state=p.S0, dfinal_state=p.dS)

    y, fin, g = run()
    keep = p.dt[t, h].clone()
    p.dt[t, h] = float("nan")
    ny, nfin, ng = run()
    assert ny[rows, h].isnan().all() and nfin[1, h].isnan().all()
    same_but(ny, y, (rows, h), "y")
    same_but(nfin, fin, (1, h), "final state")
    assert ng.ddt[t, h].isnan() and ng.dA[h].isnan() and ng.ddt_bias[h].isnan()
    same_but(ng.dx, g.dx, (slice(50, 120), h), "dx")
    same_but(ng.ddt, g.ddt, (slice(50, 120), h), "ddt")
    same_but(ng.dA, g.dA, h, "dA")
    p.dt[t, h] = float("-inf")
    iy, ifin, ig = run()
    p.dt[t, h] = -1e4
    for a, b in zip((iy, ifin, *ig), (lambda r: (r[0], r[1], *r[2]))(run())):
        assert torch.equal(a, b)
    p.dt[t, h] = keep
    p.bias[1] = float("nan")
    ny, nfin, _ = run()
    assert ny[:, 1].isnan().all() and nfin[:, 1].isnan().all()
    same_but(ny, y, (slice(None), 1), "y")


def test_nan_step_is_seen_by_one_token():
    H, P, G, N = 4, 64, 2, 64
    p = base.Problem([1] * 5, H, P, G, N, seed=25)
    start = torch.randn(5, H, P, N, device="cuda")
    ci = torch.arange(5, dtype=torch.int32, device="cuda")
    pool, bad = start.clone(), start.clone()
    y = cc.ssm_state_update(*p.args(), state_pool=pool, cache_indices=ci)
    p.dt[3, 1] = float("nan")
    ny = cc.ssm_state_update(*p.args(), state_pool=bad, cache_indices=ci)
    assert ny[3, 1].isnan().all() and bad[3, 1].isnan().all()
    same_but(ny, y, (3, 1), "y")
    same_but(bad, pool, (3, 1), "pool")


@pytest.mark.parametrize("drop", [100.0, 1e5, 1e7, 1e30])
@pytest.mark.parametrize("N", [64, 200])
def test_slow_decay_after_a_sudden_one(drop, N):
    """Tokens that drop the state (x = 0 and B = 0 there, a step of `drop`), with slow decays between them in the
    same chunk.  A decay's exponent is a sum of the steps between two rows, whatever came before them."""
    p = base.Problem([150, 64], 4, 64, 2, N, seed=26, decay=1.0)
    p.dt = p.dt.abs() * 0.1
    p.bias = torch.zeros_like(p.bias)
    for t in (10, 33, 34, 80, 150, 163):
        p.dt[t], p.x[t], p.B[t] = drop, 0, 0
    (y, fin, g), (ym, fm, gm) = p.reference(p.S0, sp=False, dy=p.dy.cpu(), dS=p.dS.cpu())
    got_fin = torch.empty_like(p.S0)
    got = cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu, dt_softplus=False, initial_state=p.S0, final_state=got_fin)
    base.close(got, y, ym, base.HALF, base.HALF, "y")
    base.close(got_fin, fin, fm, 0.0, base.FINE, "final state")
    b = cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, dt_softplus=False, initial_state=p.S0, dfinal_state=p.dS)
    for k in ("dx", "dB", "dC"):
        base.close(getattr(b, k), g[k], gm[k], base.HALF, base.HALF, k)


@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("lens,H,P,G,N", [([150, 40], 4, 64, 2, 128), ([130, 60], 6, 40, 2, 60), ([120, 70], 4, 72, 2, 200),
                                          ([1300, 90], 2, 64, 1, 64)])
def test_non_finite_x_reaches_no_earlier_row(value, lens, H, P, G, N):
    """A non-finite x makes its column of y and its row of the state non-finite from there on, and changes no other bit."""
    p = base.Problem(lens, H, P, G, N, seed=27, wide=3)
    h, c, end = 1, 37, lens[0]

    def run():
        fin = torch.empty_like(p.S0)
        return cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu, initial_state=p.S0, final_state=fin), fin

    y, fin = run()
    for t in (0, 5, 15, 16, 31, 37, 63, 64, 100, end - 1):
        keep = p.x[t, h, c].clone()
        p.x[t, h, c] = float(value)
        ny, nfin = run()
        p.x[t, h, c] = keep
        assert not ny[t:end, h, c].isfinite().any(), t
        assert not nfin[0, h, c].isfinite().any(), t
        same_but(ny, y, (slice(t, end), h, c), f"y, row {t}")
        same_but(nfin, fin, (0, h, c), f"final state, row {t}")


def test_non_finite_rows_of_B_and_C():
    """Of B: its group's heads from there on.  Of C: its group's heads in that row."""
    p = base.Problem([150, 40], 4, 64, 2, 128, seed=28)
    y = cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu)
    for t in (3, 20, 50, 77, 149):
        for which, rows in ((p.B, slice(t, 150)), (p.C, slice(t, t + 1))):
            keep = which[t, 1, 9].clone()
            which[t, 1, 9] = float("nan")
            ny = cc.ssm_scan_fwd(*p.args(), cu_seqlens=p.cu)
            which[t, 1, 9] = keep
            assert ny[rows, 2:].isnan().all()
            same_but(ny, y, (rows, slice(2, 4)), t)


@pytest.mark.parametrize("drop", [100.0, 1e5, 1e30])
@pytest.mark.parametrize("N", [64, 200])
def test_gradients_of_sudden_decays(drop, N):
    """The gradient of a step that drops the state is not its neighbours' rounding errors, and so not that times the
    step in dA."""
    p = base.Problem([150, 64], 4, 64, 2, N, seed=29, decay=1.0)
    p.dt = p.dt.abs() * 0.1
    p.bias = torch.zeros_like(p.bias)
    for t in (10, 33, 34, 80, 150, 163):
        p.dt[t], p.x[t], p.B[t] = drop, 0, 0
    (_, _, g), (_, _, gm) = p.reference(p.S0, sp=False, dy=p.dy.cpu(), dS=p.dS.cpu())
    b = cc.ssm_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, dt_softplus=False, initial_state=p.S0, dfinal_state=p.dS)
    for k in ("ddt", "dA", "ddt_bias"):
        base.close(getattr(b, k), g[k], gm[k], 0.0, base.FINE, k)
    base.close(b.dinitial_state, g["dS0"], gm["dS0"], 0.0, base.FINE, "dinitial_state")


def test_gradients_beside_much_larger_ones():
    """Small products, fast decays: a row's ddt against its own terms."""
    p = base.Problem([1100, 127, 200, 200], 4, 1, 2, 1, seed=936630773, dt32=True, decay=30.0, step=1.0)
    base.check_bwd(p, p.S0, p.dS)


@pytest.mark.parametrize("rows,seqlen", [(4096, 4096), (4096, 1024)])
def test_decay_rate_gradient_has_no_offset(rows, seqlen):
    """dA is odd in dy.  Where x, B and C have a mean, an offset of the adjoints adds up in it over all rows while its
    own terms cancel.  A term's four factors (step, decay, state, adjoint) are off by 2^-24 at most: 2^-22 a call if all
    rows were off the same way, twice that for two calls."""
    print(f"[gpu] offset of dA, {rows} rows of {seqlen}", flush=True)
    H, P, N = 32, 64, 128
    gen = torch.Generator().manual_seed(30)

    def rnd(*shape):
        return torch.nn.functional.silu(torch.randn(shape, generator=gen)).bfloat16().cuda()

    x, B, C = rnd(rows, H, P), rnd(rows, 1, N), rnd(rows, 1, N)
    dt = (0.02 * (1 + torch.rand(rows, H, generator=gen))).cuda()
    A = -torch.linspace(0.2, 3, H).cuda()
    dy = torch.randn(rows, H, P, generator=gen).bfloat16().cuda()
    up, down = [cc.ssm_scan_bwd(s * dy, x, dt, A, B, C, seqlen=seqlen, dt_softplus=False).dA.double() for s in (1, -1)]
    assert (up + down).norm() <= 2.0 ** -21 * up.norm(), float((up + down).norm() / up.norm())
