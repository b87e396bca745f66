"""GPU: the layer norm against float64, forward and backward, alone and of a residual's sum.

Tolerances count roundings: a bf16 result 2^-8 of its value; FP32 sums of at most 32768 channels by 64 or more threads, 8
or 32 terms a thread and ten steps of a tree, so at most 42 roundings of 2^-24 each: 2^-18 of the terms' magnitudes; a sum
over rows: at most 600 terms: 2^-14.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import causal_depthwise_conv1d_width_amd as cc  # noqa: E402

bf16, f32 = torch.bfloat16, torch.float32
EPS = 1e-5


def within(got, want, allowed, what):
    got = got.detach().double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    excess = (got - want).abs() - allowed - 1e-30
    assert excess.max() <= 0, f"{what}: off by {float((got - want).abs().flatten()[int(excess.argmax())]):.3g}"


def make(rows, d, seed, mean=0.0, wide=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, dtype=bf16):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    x, dy = (rnd(rows, d + wide)[:, :d] for _ in range(2))
    return (x + mean if mean else x), dy, 1 + 0.1 * rnd(d, dtype=f32), 0.1 * rnd(d, dtype=f32), rnd


CASES = [(1, 1), (3, 2), (64, 2055), (5, 512), (7, 513), (130, 300), (600, 2048), (2, 8193), (3, 20001), (2, 32768)]


@pytest.mark.parametrize("rows,d", CASES)
@pytest.mark.parametrize("kind", ["plain", "bf16", "fp32"])
def test_forward_and_backward(rows, d, kind):
    x, dy, w, bias, rnd = make(rows, d, rows + d, mean=0.0 if kind == "plain" else 3.0, wide=3 if kind == "fp32" else 0)
    wt = bf16 if kind == "bf16" else f32
    w, bias = w.to(wt), bias.to(wt)
    scale, res, dr = 1.0, None, None
    if kind != "plain":
        scale, res = 0.7, rnd(rows, d, dtype=f32 if kind == "fp32" else bf16)
        dr = rnd(rows, d, dtype=res.dtype)
    y, r = cc.layer_norm_fwd(x, w, bias, residual=res, scale=scale)
    h = x
    if res is not None:
        want = res.double() + scale * x.double()
        step = 2.0 ** -8 if kind == "bf16" else 2.0 ** -23
        within(r, want, step * want.abs() + 2.0 ** -23 * (res.double().abs() + x.double().abs()), "residual_out")
        h = r
    else:
        assert r is None
    h64 = h.double().requires_grad_()
    w64, b64 = w.double().requires_grad_(), bias.double().requires_grad_()
    c = h64 - h64.mean(-1, keepdim=True)
    inv = torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS)
    out = c * inv * w64 + b64
    with torch.no_grad():  # an error of 2^-18 of the row's largest value in the mean, through to the result
        noise = 2.0 ** -18 * h64.abs().amax(-1, keepdim=True) * inv * (1 + (c * inv).abs())
    within(y, out, 2.0 ** -8 * out.abs() + 2.0 ** -18 * (c * inv * w64).abs() + noise * w64.abs(), "y")
    g = cc.layer_norm_bwd(dy, h, w, residual=res is not None, dresidual_out=dr, scale=scale)
    gh, gw, gb = torch.autograd.grad(out, [h64, w64, b64], dy.double())
    dh = (dy.double() * w64).abs()
    terms = inv * (dh + dh.mean(-1, keepdim=True) + (c * inv).abs() * (dh * (c * inv).abs()).mean(-1, keepdim=True))
    fine = 2.0 ** -17 * terms + 4 * noise * inv * dh.amax(-1, keepdim=True)
    if dr is not None:
        gh = gh + dr.double()
        step = 2.0 ** -8 if kind == "bf16" else 2.0 ** -22
        within(g.dresidual, gh, step * gh.abs() + fine + 2.0 ** -22 * dr.double().abs(), "dresidual")
    else:
        assert g.dresidual is None
    within(g.dx, scale * gh, 2.0 ** -8 * (scale * gh).abs() + fine + 2.0 ** -22 * gh.abs(), "dx")
    per_row = dy.double().abs()
    within(g.dweight, gw, (2.0 ** -14 * per_row * (c * inv).abs() + noise * per_row).sum(0), "dweight")
    within(g.dbias, gb, 2.0 ** -14 * per_row.sum(0), "dbias")


def test_gradient_against_differences():
    """d(sum dy y) along a direction, by central differences in float64 of the formula, against the kernel's gradient."""
    rows, d = 6, 96
    x, dy, w, bias, rnd = make(rows, d, 5)
    g = cc.layer_norm_bwd(dy, x, w)
    e = rnd(rows, d).double()

    def loss(h):
        c = h - h.mean(-1, keepdim=True)
        return (dy.double() * (c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * w.double() + bias.double())).sum()

    t = 1e-5
    slope = (loss(x.double() + t * e) - loss(x.double() - t * e)) / (2 * t)
    # each dx is rounded by 2^-8 of itself; differences are exact to t^2
    assert abs(float((g.dx.double() * e).sum() - slope)) <= float(2.0 ** -8 * (g.dx.double() * e).abs().sum()) + 1e-6


def test_large_mean():
    """The variance is that of the centred values: a mean of 1000 standard deviations costs its own rounding only."""
    rows, d = 16, 1000
    res = (1000.0 + torch.randn(rows, d, device="cuda"))
    x = torch.zeros(rows, d, dtype=bf16, device="cuda")
    w = torch.ones(d, device="cuda")
    y, r = cc.layer_norm_fwd(x, w, residual=res)
    h = r.double()
    want = (h - h.mean(-1, keepdim=True)) / torch.sqrt(h.var(-1, correction=0, keepdim=True) + EPS)
    within(y, want, 2.0 ** -8 * want.abs() + 2.0 ** -18 * 1000 * (1 + want.abs()), "y")


def test_in_place_and_bits():
    rows, d = 40, 600
    x, dy, w, bias, rnd = make(rows, d, 8)
    res = rnd(rows, d, dtype=f32)
    y, r = cc.layer_norm_fwd(x, w, bias, residual=res, scale=0.5)
    mine = res.clone()
    y2, r2 = cc.layer_norm_fwd(x, w, bias, residual=mine, residual_out=mine, scale=0.5)
    assert r2 is mine and torch.equal(mine, r) and torch.equal(y, y2)
    dr = rnd(rows, d, dtype=f32)
    a = cc.layer_norm_bwd(dy, r, w, residual=True, dresidual_out=dr, scale=0.5)
    own = dr.clone()
    ws = torch.full((cc.layer_norm_bwd_workspace_bytes(rows, d),), 0xff, dtype=torch.uint8, device="cuda")
    b = cc.layer_norm_bwd(dy, r, w, residual=True, dresidual_out=own, dresidual=own, scale=0.5, workspace=ws)
    assert all(torch.equal(s, t) for s, t in zip(a, b)) and b.dresidual is own
    none = cc.layer_norm_bwd(dy, r, w, residual=True, scale=0.5)
    zero = cc.layer_norm_bwd(dy, r, w, residual=True, dresidual_out=torch.zeros_like(r), scale=0.5)
    assert all(torch.equal(s, t) for s, t in zip(none, zero))


def test_no_rows_and_not_finite():
    w = torch.ones(50, device="cuda")
    empty = torch.empty(0, 50, dtype=bf16, device="cuda")
    y, r = cc.layer_norm_fwd(empty, w)
    assert y.shape == (0, 50) and r is None
    y, r = cc.layer_norm_fwd(empty, w, residual=empty.float())
    assert r.shape == (0, 50)
    g = cc.layer_norm_bwd(empty, empty, w)
    assert (g.dweight == 0).all() and (g.dbias == 0).all() and g.dx.shape == (0, 50)
    x = torch.randn(5, 50, device="cuda").to(bf16)
    clean = cc.layer_norm_fwd(x, w)[0]
    x[2, 7] = float("inf")
    y = cc.layer_norm_fwd(x, w)[0]
    rest = [0, 1, 3, 4]
    assert torch.equal(y[rest], clean[rest]) and torch.isnan(y[2]).all()


def test_captured():
    rows, d = 33, 700
    x, dy, w, bias, rnd = make(rows, d, 4)
    res, dr = rnd(rows, d, dtype=f32), rnd(rows, d, dtype=f32)

    def work():
        y, r = cc.layer_norm_fwd(x, w, bias, residual=res)
        return y, r, *cc.layer_norm_bwd(dy, r, w, residual=True, dresidual_out=dr)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for _ in range(3):
        x.mul_(1.5)
        res.add_(0.1)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        assert all(torch.equal(a, b) for a, b in zip(got, work()))
