"""GPU: the gated delta rule's backward against float64 (delta_reference.py).

Tolerances count roundings.  A bf16 result: 2^-8 of its value.  dq and dk: the decayed scores of their terms between two
rows once more, 2^-8 (1 + 2^-6) of these terms' magnitudes.  Everything else is FP32 arithmetic on operands of two fp16
parts, off by at most 2^-23 of their column's, row's or tile's largest (two roundings of 2^-24; at most eight such operands
a chunk): with at most 40 roundings of 2^-24 a chunk in a state or an adjoint, as many in the other and in the products of
both, over at most 8 chunks, 2^-14 of the largest sum of magnitudes in the head (ddt, db, the initial states' gradient); of dA and
d(dt_bias) of their sum over rows; the same share of the largest |adjoint| |key| or |state| |key| stays in dq, dk, dv.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import causal_depthwise_conv1d_width_amd as cc  # noqa: E402
import delta_reference as ref  # noqa: E402
from test_gpu_delta import HALF, SHAPES, Problem, within  # noqa: E402

bf16, f32 = torch.bfloat16, torch.float32
FINE = 2.0 ** -14


def reference(p, S0=None, dS=None, args=None):
    n = {"qk_norm": "norm", "beta_max": "beta", "norm_eps": "eps", "dt_softplus": "softplus", "scale": "scale"}
    H, P, _, N = p.dims
    zero = torch.zeros(len(p.lens), H, P, N)
    return ref.gradients(*((t.cpu() if t is not None else None) for t in (args or p.args())), p.bounds,
                         zero if S0 is None else S0.cpu(), p.dy.cpu(), None if dS is None else dS.cpu(),
                         **{n[m]: x for m, x in p.kw.items()})


def check(p, got, want):
    g, m = want
    rows = [t for s, e in p.bounds for t in range(s, e)]
    gate = 2.0 ** -8 if p.dt.dtype is bf16 else 0.0
    if rows:
        top = m["dl"][rows].amax(0)  # a head's largest sum
        for name in ("dq", "dk", "dv"):
            w = g[name][rows]
            extra = HALF * m[name][rows] if name != "dv" else 0.0
            within(getattr(got, name)[rows], w, 2.0 ** -8 * w.abs() + extra + FINE * w.abs().amax((0, 2), keepdim=True), name)
        w = g["ddt"][rows]
        within(got.ddt[rows], w, gate * w.abs() + FINE * m["slope"][rows] * top, "ddt")
        w = g["db"][rows]
        within(got.db[rows], w, gate * w.abs() + FINE * m["db"][rows].amax(0), "db")
        within(got.dA, g["dA"], FINE * (m["step"][rows] * top).sum(0), "dA")
        if got.ddt_bias is not None:
            within(got.ddt_bias, g["ddt_bias"], FINE * (m["slope"][rows] * top).sum(0), "ddt_bias")
    if got.dinitial_state is not None:
        within(got.dinitial_state, g["dS0"], FINE * m["dS0"].amax(-1, keepdim=True), "dinitial_state")


@pytest.mark.parametrize("lens,H,P,G,N", SHAPES, ids=str)
@pytest.mark.parametrize("kind", ["norm", "raw"])
def test_gradients(lens, H, P, G, N, kind):
    p = Problem(lens, H, P, G, N, seed=len(lens) + N, norm=kind == "norm", beta=1.0 if kind == "norm" else 1.5,
                gates=f32 if kind == "norm" else bf16, wide=5 if kind == "raw" else 0, key=0.8 if kind == "raw" else 1.0)
    check(p, cc.delta_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, **p.kw), reference(p))
    g = cc.delta_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, initial_state=p.S0, dfinal_state=p.dS, **p.kw)
    check(p, g, reference(p, p.S0, p.dS))


@pytest.mark.parametrize("kw", [dict(scale=1.0), dict(dt_softplus=False), dict(norm_eps=0.1), dict(beta=2.0)], ids=str)
def test_options(kw):
    p = Problem([90, 20], 2, 32, 1, 48, seed=3, **kw)
    if "dt_softplus" in kw:
        p.dt = p.dt.abs() * 0.2
        p.bias = p.bias.abs() * 0.1
    check(p, cc.delta_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, **p.kw), reference(p))
    args = (*p.args()[:6], None)
    g = cc.delta_scan_bwd(p.dy, *args, cu_seqlens=p.cu, dfinal_state=p.dS, **p.kw)
    assert g.ddt_bias is None and g.dinitial_state is None
    check(p, g, reference(p, None, p.dS, args))


def test_correlated_keys():
    p = Problem([128], 2, 64, 1, 64, seed=9, beta=2.0, decay=0.01, key=0.05)
    p.k.add_(1.0)
    p.b.add_(3.0)
    check(p, cc.delta_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, **p.kw), reference(p))


def test_sudden_decays():
    """Rows that forget almost everything among slow ones: dl of the slow rows loses nothing to the sums beside them."""
    p = Problem([150], 2, 32, 1, 32, seed=33, decay=0.01)
    p.dt[[20, 21, 70, 130]] = 4000.0
    check(p, cc.delta_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, **p.kw), reference(p))


def test_no_rates_and_no_rows():
    """b = -inf: no write and no gradient of b; no rows; sequences without rows pass their adjoint on."""
    p = Problem([70], 2, 16, 1, 32, seed=41)
    p.b[5:20] = -float("inf")
    g = cc.delta_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, **p.kw)
    assert (g.db[5:20] == 0).all() and (g.dv[5:20] == 0).all()
    check(p, g, reference(p))
    e = Problem([0, 0], 2, 16, 1, 16, seed=2)
    g = cc.delta_scan_bwd(e.dy, *e.args(), cu_seqlens=e.cu, initial_state=e.S0, dfinal_state=e.dS, **e.kw)
    assert torch.equal(g.dinitial_state, e.dS) and (g.dA == 0).all() and (g.ddt_bias == 0).all()
    g = cc.delta_scan_bwd(e.dy, *e.args(), cu_seqlens=e.cu[:1], **e.kw)
    assert (g.dA == 0).all() and g.dq.shape == (0, 1, 16)


def test_ranges_of_one_gradient_array():
    """dq, dk, dv side by side; rows outside the sequences and the columns between stay."""
    p = Problem([60, 50], 4, 24, 2, 40, seed=51, pad=4, first=3)
    H, P, G, N = p.dims
    row = torch.full((p.R, 2 * G * N + H * P + 6), 7.0, dtype=bf16, device="cuda")
    gates = torch.full((p.R, 2 * H + 1), 7.0, device="cuda")
    dq, dk = row[:, :G * N].view(p.R, G, N), row[:, G * N:2 * G * N].view(p.R, G, N)
    dv = row[:, 2 * G * N:2 * G * N + H * P].view(p.R, H, P)
    g = cc.delta_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, dq=dq, dk=dk, dv=dv, ddt=gates[:, :H], db=gates[:, H:2 * H], **p.kw)
    check(p, g, reference(p))
    assert (row[:, -6:] == 7).all() and (row[:3] == 7).all() and (row[-4:] == 7).all()
    assert (gates[:, -1] == 7).all() and (gates[:3] == 7).all() and (gates[-4:] == 7).all()
    for t in (p.q, p.k, p.v, p.dt, p.b, p.dy):
        t[:3] = float("nan")
        t[-4:] = float("inf")
    again = cc.delta_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, **p.kw)
    for name in ("dq", "dk", "dv", "ddt", "db"):
        assert torch.equal(getattr(again, name)[3:-4], getattr(g, name)[3:-4]), name
    assert torch.equal(again.dA, g.dA)


@pytest.mark.parametrize("where", ["v", "k", "q", "dt", "b", "dy"])
def test_not_finite_stays_in_sequence_and_group(where):
    p = Problem([100, 30], 4, 20, 2, 40, seed=13)
    clean = cc.delta_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, **p.kw)
    t = dict(v=p.v, k=p.k, q=p.q, dt=p.dt, b=p.b, dy=p.dy)[where]
    if t.dim() == 3:
        t[70, 1 if where in "qk" else 2, 3] = float("nan")
    else:
        t[70, 2] = float("nan")
    g = cc.delta_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, **p.kw)
    for name, heads in (("dq", slice(0, 1)), ("dk", slice(0, 1)), ("dv", slice(0, 2)), ("ddt", slice(0, 2)), ("db", slice(0, 2))):
        a, b = getattr(g, name), getattr(clean, name)
        assert torch.equal(a[100:], b[100:]) and torch.equal(a[:, heads], b[:, heads]), name
    assert torch.equal(g.dA[:2], clean.dA[:2]) and not torch.isfinite(g.dA[2:]).all()
    assert not torch.isfinite(g.dk[:100, 1]).all()


def test_same_bits_any_workspace_and_stream():
    p = Problem([90, 70, 200], 4, 64, 2, 128, seed=23)
    kw = dict(cu_seqlens=p.cu, initial_state=p.S0, dfinal_state=p.dS, **p.kw)
    a = cc.delta_scan_bwd(p.dy, *p.args(), **kw)
    need = cc.delta_scan_bwd_workspace_bytes(p.v, p.k, p.dt, 3)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = cc.delta_scan_bwd(p.dy, *p.args(), workspace=ws[16:16 + need], stream=s, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert (ws[:16] == 0xff).all() and (ws[16 + need:] == 0xff).all()


def test_captured():
    """Forward and backward in one graph, replayed with new inputs between eager work."""
    p = Problem([60, 85], 2, 32, 1, 64, seed=29)

    def work():
        y = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, initial_state=p.S0, **p.kw)
        return y, *cc.delta_scan_bwd(y, *p.args(), cu_seqlens=p.cu, initial_state=p.S0, **p.kw)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for _ in range(3):
        p.v.mul_(-0.5)
        p.k.add_(0.25)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        assert all(torch.equal(a, b) for a, b in zip(got, work()))
        torch.randn(1000, device="cuda").sum().item()
