"""GPU: the norms around a mixer block against float64 (ssm_reference.py).

bf16 results are rounded once from FP32 arithmetic: 2^-8 of the value, and 2^-16 of the row's scale for
the FP32 sums (hardware exp2, reciprocal and rsqrt about 1 ulp each).  FP32 results (dw, FP32 residuals)
see the arithmetic only: 2^-16 of the scale of their terms.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import causal_depthwise_conv1d_width_amd as cc  # noqa: E402
import ssm_reference as ref  # noqa: E402

FINE = 2.0 ** -16


def rnd(gen, *shape, dtype=torch.bfloat16, wide=0):
    t = torch.randn(shape[0], shape[1] + wide, generator=gen).to(dtype).cuda()
    return t[:, wide // 2:wide // 2 + shape[1]]


def close(got, want, scale, what):
    own = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    got = got.cpu().double()
    assert torch.isfinite(got).all(), what
    excess = (got - want).abs() - (own * want.abs() + FINE * scale + 1e-30)
    assert excess.numel() == 0 or excess.max() <= 0, f"{what}: {float((got - want).abs().max()):.3g}"


def row_scale(t, extra=0.0):
    """Per row: the largest magnitude, the scale of the row's reductions."""
    return t.abs().amax(-1, keepdim=True) * 4 + extra


CASES = [(1, 1, 1), (3, 8, 8), (5, 1000, 500), (64, 4096, 1024), (7, 2055, 2055), (130, 2048, 256), (9, 5000, 5000),
         (4, 9000, 9000), (2, 32768, 32768), (700, 96, 32), (0, 64, 64)]


@pytest.mark.parametrize("rows,d,group", CASES)
@pytest.mark.parametrize("norm_first", [False, True])
@pytest.mark.parametrize("w32", [True, False])
def test_gated(rows, d, group, norm_first, w32):
    print(f"[gpu] gated {rows}x{d}/{group} {norm_first} {w32}", flush=True)
    gen = torch.Generator().manual_seed(rows + d)
    x, z, dy = rnd(gen, rows, d, wide=3), rnd(gen, rows, d), rnd(gen, rows, d, wide=8)
    w = (1 + 0.1 * torch.randn(d, generator=gen)).to(torch.float32 if w32 else torch.bfloat16).cuda()
    kw = dict(group_size=group, norm_before_gate=norm_first, eps=1e-5)
    y = cc.gated_norm_fwd(x, z, w, **kw)
    dx, dz, dw = cc.gated_norm_bwd(dy, x, z, w, **kw)
    torch.cuda.synchronize()
    ry, rx, rz, rw = ref.gated(x.cpu(), z.cpu(), w.cpu(), group, norm_first, 1e-5, dy.cpu())
    if rows == 0:
        assert not dw.any()
        return
    close(y, ry, row_scale(ry), "y")
    # d(u) = (d n's gradient - its mean parts) / rms: its FP32 error is that of the gradients over the rms
    u = x.cpu().double() * (1 if norm_first else z.cpu().double() * torch.sigmoid(z.cpu().double()))
    inv = torch.rsqrt(u.view(rows, -1, group).square().mean(-1) + 1e-5).amax(-1, keepdim=True)
    scale = row_scale(rx) + dy.cpu().double().abs().amax() * (1 + inv)
    close(dx, rx, scale, "dx")
    close(dz, rz, row_scale(rz) + scale * x.cpu().double().abs().amax(), "dz")
    terms = (dy.cpu().double() * ry).abs().sum(0) + ry.abs().sum(0) + dy.cpu().double().abs().sum(0)
    close(dw, rw, terms, "dw")


@pytest.mark.parametrize("rows,d", [(1, 1), (3, 8), (64, 2055), (33, 2048), (5, 6001), (2, 20000), (1030, 100), (0, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("in_place", [False, True])
def test_residual(rows, d, dtype, in_place):
    print(f"[gpu] residual {rows}x{d} {dtype} {in_place}", flush=True)
    gen = torch.Generator().manual_seed(rows + d)
    x, r, dy = rnd(gen, rows, d), rnd(gen, rows, d, dtype=dtype, wide=2), rnd(gen, rows, d)
    dr = rnd(gen, rows, d, dtype=dtype)
    w = (1 + 0.1 * torch.randn(d, generator=gen)).cuda()
    ry, rr, rx, rd, rw = ref.residual(x.cpu(), r.cpu(), w.cpu(), 0.25, 1e-6, dy.cpu(), dr.cpu())
    y, total = cc.residual_norm_fwd(x, r, w, scale=0.25, eps=1e-6, residual_out=r if in_place else None)
    assert not in_place or total is r
    # 0.25 x + r: exact products, one FP32 rounding, then the stored type's
    assert torch.equal(total.cpu(), rr.float().to(dtype))
    dx, dres, dw = cc.residual_norm_bwd(dy, dr, total, w, scale=0.25, eps=1e-6, dresidual=dr if in_place else None)
    torch.cuda.synchronize()
    if rows == 0:
        assert not dw.any()
        return
    scale = row_scale(rd) + dy.cpu().double().abs().amax() * 4
    # a row's gradient is divided by its rms, which may be small at d = 1
    scale = scale / rr.square().mean(-1, keepdim=True).sqrt().clamp(max=1.0)
    close(y, ry, row_scale(ry), "y")
    close(dx, rx, scale, "dx")
    close(dres, rd, scale, "dresidual")
    close(dw, rw, (dy.cpu().double() * ry).abs().sum(0) + dy.cpu().double().abs().sum(0), "dw")


def test_residual_without_other_gradient():
    gen = torch.Generator().manual_seed(1)
    r, dy = rnd(gen, 40, 513, dtype=torch.float32), rnd(gen, 40, 513)
    w = torch.ones(513, device="cuda")
    a = cc.residual_norm_bwd(dy, None, r, w)
    b = cc.residual_norm_bwd(dy, torch.zeros_like(r), r, w)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_zero_rows_have_no_nan():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, device="cuda")
    dy = torch.ones_like(x)
    assert not cc.gated_norm_fwd(x, x, w).any()
    for t in cc.gated_norm_bwd(dy, x, x, w):
        assert torch.isfinite(t).all()
    # the largest gates: silu(z) = z or 0, its slope 1 or 0
    z = torch.tensor([[-3e38, 3e38, -200.0, 200.0]], dtype=torch.bfloat16, device="cuda")
    x = torch.tensor([[1.0, 1e-38, 1.0, 1.0]], dtype=torch.bfloat16, device="cuda")
    y = cc.gated_norm_fwd(x, z, torch.ones(4, device="cuda"))
    assert torch.isfinite(y).all() and float(y[0, 3]) == 2.0


def test_same_bits_graph_and_stream():
    gen = torch.Generator().manual_seed(2)
    x, z, dy = rnd(gen, 3000, 1024), rnd(gen, 3000, 1024), rnd(gen, 3000, 1024)
    w = torch.randn(1024, generator=gen).cuda()
    first = cc.gated_norm_bwd(dy, x, z, w, group_size=256)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (None, side):
        torch.cuda.synchronize()
        again = cc.gated_norm_bwd(dy, x, z, w, group_size=256, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cc.gated_norm_bwd(dy, x, z, w, group_size=256)
        y, r = cc.residual_norm_fwd(x, z, w)
    for _ in range(3):
        x.mul_(0.5)
        want = cc.gated_norm_bwd(dy, x, z, w, group_size=256)
        wy, wr = cc.residual_norm_fwd(x, z, w)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*out, y, r), (*want, wy, wr)))
