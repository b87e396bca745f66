"""Refusals of the scan, step and norm entry points, decided on the host (CPU only): the C ABI's by fake
addresses that are compared and never read, the torch binding's by host tensors."""
import ctypes
import os
import re

import pytest

from causal_depthwise_conv1d_width_amd import _lib

torch = pytest.importorskip("torch")

import causal_depthwise_conv1d_width_amd as cc  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EWORKSPACE = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from causal_depthwise_conv1d_width_amd.build import build
        build()
    return _lib.load_ssm()


def test_header_and_binding_agree(lib):
    text = open(os.path.join(ROOT, "include", "ssm.h")).read()
    names = set(re.findall(r"^(?:int|size_t)\s+(\w+)\s*\(", text, re.M))
    assert names == set(_lib.SSM_SIGNATURES)
    for n in names:
        assert hasattr(lib, n)


class Call:
    """Arguments of one entry point at fake, disjoint addresses, changed by name."""

    def __init__(self):
        self.next = 1 << 40

    def at(self, nbytes):
        p = self.next
        self.next += (nbytes + 4096 + 255) // 256 * 256
        return p

    def scan(self, lib, bwd=False, **kw):
        R, H, P, G, N, nseq = kw.get("rows", 100), kw.get("H", 4), kw.get("P", 64), kw.get("G", 2), kw.get("N", 64), 3
        hp, gn, big = H * P, G * N, 1 << 22
        sh = _lib.SsmShape(H, P, G, N, kw.get("dt_dtype", 1), kw.get("softplus", 1))
        v = {k: self.at(big) for k in ("dy", "x", "dt", "A", "B", "C", "D", "bias", "y", "S0", "dS", "dx", "ddt", "dA",
                                       "dB", "dC", "dD", "db", "dS0", "cu", "ci", "hi", "fin")}
        v.update(dy_ld=hp, x_ld=hp, dt_ld=H, B_ld=gn, C_ld=gn, y_ld=hp, dx_ld=hp, ddt_ld=H, dB_ld=gn, dC_ld=gn,
                 seq_idx=None, seqlen=0, ws=self.at(1 << 30), ws_bytes=1 << 30, slots=8, s_slot=hp * N)
        v.update({k: (v[x] if isinstance(x, str) else x) for k, x in kw.items()})
        seq = _lib.Seq(v["cu"], nseq, v["seq_idx"], v["seqlen"])
        q = None if kw.get("no_seq") else ctypes.byref(seq)
        if bwd:
            return lib.ssm_scan_bwd(ctypes.byref(sh), R, v["dy"], v["dy_ld"], v["x"], v["x_ld"], v["dt"], v["dt_ld"], v["A"],
                                    v["B"], v["B_ld"], v["C"], v["C_ld"], v["D"], v["bias"], q, v["S0"], v["dS"],
                                    v["dx"], v["dx_ld"], v["ddt"], v["ddt_ld"], v["dA"], v["dB"], v["dB_ld"], v["dC"],
                                    v["dC_ld"], v["dD"], v["db"], v["dS0"], v["ws"], v["ws_bytes"], None)
        st = _lib.SsmStates(v.get("initial", v["S0"]), v["fin"], v["slots"], v["s_slot"], v["ci"], v["hi"])
        if kw.get("step"):
            return lib.ssm_state_update(ctypes.byref(sh), R, v["x"], v["x_ld"], v["dt"], v["dt_ld"], v["A"], v["B"], v["B_ld"],
                                        v["C"], v["C_ld"], v["D"], v["bias"], ctypes.byref(st), v["y"], v["y_ld"], None)
        return lib.ssm_scan_fwd(ctypes.byref(sh), R, v["x"], v["x_ld"], v["dt"], v["dt_ld"], v["A"], v["B"], v["B_ld"],
                                v["C"], v["C_ld"], v["D"], v["bias"], q, ctypes.byref(st), v["y"], v["y_ld"], v["ws"],
                                v["ws_bytes"], None)


SHARED = [dict(H=0), dict(P=0), dict(G=3), dict(N=0), dict(N=257), dict(rows=-1), dict(dt_dtype=2), dict(softplus=2),
          dict(no_seq=True), dict(seq_idx=4096), dict(cu=None, seqlen=0), dict(cu=None, seqlen=33), dict(x_ld=10),
          dict(B_ld=10), dict(C_ld=10), dict(dt_ld=3), dict(A=None), dict(x=None), dict(dt=None), dict(B=None),
          dict(x=(1 << 40) + 1), dict(dt=(1 << 40) + 2), dict(x_ld=1 << 47), dict(ws=(1 << 45) + 8)]
FWD = [dict(y=None), dict(y_ld=1), dict(y="x"), dict(y="B"), dict(y="cu"), dict(y="D"), dict(fin="x"), dict(fin="y"),
       dict(slots=0), dict(s_slot=5), dict(ci=None, slots=2), dict(initial=None, fin=None), dict(y="S0"), dict(y="ci")]
BWD = [dict(dy=None), dict(dx=None), dict(dA=None), dict(dB=None), dict(dy_ld=1), dict(dx_ld=1), dict(ddt_ld=1),
       dict(dx="dy"), dict(dx="x"), dict(dB="dC"), dict(dS0="dS"), dict(dA="dD"), dict(db="cu"), dict(ws="x"), dict(ddt="dt")]


@pytest.mark.parametrize("kw", SHARED + FWD, ids=str)
def test_scan_forward_refuses(lib, kw):
    kw = dict(kw, rows=4000) if "ws" in kw else kw  # a call that needs a workspace
    assert Call().scan(lib, **kw) == EINVAL


@pytest.mark.parametrize("kw", SHARED + BWD, ids=str)
def test_scan_backward_refuses(lib, kw):
    assert Call().scan(lib, bwd=True, **kw) == EINVAL


def test_workspaces(lib):
    assert Call().scan(lib, bwd=True, ws_bytes=0) == EWORKSPACE
    assert Call().scan(lib, bwd=True, ws=None) == EWORKSPACE
    assert Call().scan(lib, rows=9000, H=1, G=1, ws_bytes=100) == EWORKSPACE
    sh = _lib.SsmShape(4, 64, 2, 128, 1, 1)
    assert lib.ssm_scan_fwd_workspace_bytes(ctypes.byref(sh), 64, 2) == 0
    assert lib.ssm_scan_fwd_workspace_bytes(ctypes.byref(sh), 100000, 1) > 0
    # two states of 64 x 128 FP32 values a chunk and head, at least
    assert lib.ssm_scan_bwd_workspace_bytes(ctypes.byref(sh), 640, 1) >= 2 * 10 * 4 * 64 * 128 * 4
    assert lib.ssm_scan_bwd_workspace_bytes(ctypes.byref(_lib.SsmShape(4, 64, 3, 128, 1, 1)), 640, 1) == 0
    assert lib.norm_bwd_workspace_bytes(10, 100, 33) == 0
    assert lib.norm_bwd_workspace_bytes(10, 100, 50) >= 100 * 4


@pytest.mark.parametrize("kw", [dict(N=257), dict(x=None), dict(A=None), dict(y_ld=1), dict(ci=None), dict(initial=None),
                                dict(y="x"), dict(y="ci"), dict(y="S0"), dict(slots=0), dict(s_slot=1), dict(rows=-1),
                                dict(dt_ld=1)], ids=str)
def test_step_refuses(lib, kw):
    kw = dict(kw)
    c = Call()
    pool = c.at(1 << 22)
    base = dict(S0=pool, fin=pool, step=True)
    base.update(kw)
    if kw.get("y") == "S0":
        base["y"] = pool
    assert c.scan(lib, **base) == EINVAL


def test_interleaved_columns_are_not_an_overlap(lib):
    """Column ranges of one wider array may be read and written side by side; shared columns may not."""
    c = Call()
    row = c.at(1 << 24)
    ld = 4 * 64 + 2 * 64 * 2
    side = dict(dx=row, dx_ld=ld, dB=row + 2 * 256, dB_ld=ld, dC=row + 2 * (256 + 128), dC_ld=ld)
    assert c.scan(lib, bwd=True, ws_bytes=0, **side) == EWORKSPACE  # past every other check's first half
    assert c.scan(lib, bwd=True, **dict(side, dC=row + 2 * (256 + 127))) == EINVAL
    assert c.scan(lib, bwd=True, **dict(side, dx=row + 2)) == EINVAL


def norm(lib, c, which, **kw):
    v = dict(rows=10, d=96, group=32, x=c.at(1 << 20), z=c.at(1 << 20), w=c.at(1 << 16), y=c.at(1 << 20), dy=c.at(1 << 20),
             dx=c.at(1 << 20), dz=c.at(1 << 20), dw=c.at(1 << 16), r=c.at(1 << 20), ro=c.at(1 << 20), dr=c.at(1 << 20),
             ws=c.at(1 << 24), ws_bytes=1 << 24, ld=96, eps=1e-5, wd=1, rt=1)
    v.update({k: (v[x] if isinstance(x, str) else x) for k, x in kw.items()})
    R, d, ld = v["rows"], v["d"], v["ld"]
    if which == "gated_fwd":
        return lib.gated_norm_fwd(R, d, v["group"], v["x"], ld, v["z"], ld, v["w"], v["wd"], 0, v["eps"], v["y"], ld, None)
    if which == "gated_bwd":
        return lib.gated_norm_bwd(R, d, v["group"], v["dy"], ld, v["x"], ld, v["z"], ld, v["w"], v["wd"], 0, v["eps"], v["dx"],
                                  ld, v["dz"], ld, v["dw"], v["ws"], v["ws_bytes"], None)
    if which == "residual_fwd":
        return lib.residual_norm_fwd(R, d, v["x"], ld, v["r"], ld, v["rt"], 1.0, v["w"], v["wd"], v["eps"], v["y"], ld, v["ro"],
                                     ld, None)
    return lib.residual_norm_bwd(R, d, v["dy"], ld, v["dr"], ld, v["r"], ld, v["rt"], 1.0, v["w"], v["wd"], v["eps"], v["dx"],
                                 ld, v["ro"], ld, v["dw"], v["ws"], v["ws_bytes"], None)


@pytest.mark.parametrize("which,kw", [(w, kw) for w, own in {
    "gated_fwd": [dict(group=33), dict(group=0), dict(x=None), dict(z=None), dict(y=None), dict(y="x"), dict(y="z"), dict(y="w"),
                  dict(d=65536, group=65536, ld=65536)],
    "gated_bwd": [dict(group=33), dict(dy=None), dict(dx="dy"), dict(dx="dz"), dict(dw=None), dict(ws="x"), dict(dw="w")],
    "residual_fwd": [dict(rt=2), dict(r=None), dict(ro="x"), dict(y="ro"), dict(y="r"), dict(ro=None)],
    "residual_bwd": [dict(rt=2), dict(r=None), dict(ro="r"), dict(dx="ro"), dict(dx="dr"), dict(dw=None), dict(ws="dr")],
}.items() for kw in own + [dict(rows=-1), dict(d=0), dict(w=None), dict(wd=2), dict(ld=95), dict(eps=-1.0), dict(eps=float("nan"))]],
    ids=str)
def test_norms_refuse(lib, which, kw):
    assert norm(lib, Call(), which, **kw) == EINVAL


def test_norm_workspaces(lib):
    for which in ("gated_bwd", "residual_bwd"):
        assert norm(lib, Call(), which, ws_bytes=4) == EWORKSPACE
        assert norm(lib, Call(), which, ws=None) == EWORKSPACE


# ------------------------------------------------------------------ the torch binding
def tensors(R=8, H=2, P=16, G=1, N=16):
    bf = torch.bfloat16
    return (torch.zeros(R, H, P, dtype=bf), torch.zeros(R, H), torch.zeros(H), torch.zeros(R, G, N, dtype=bf),
            torch.zeros(R, G, N, dtype=bf))


def test_host_tensors_are_refused():
    x, dt, A, B, C = tensors()
    pool = torch.zeros(9, 2, 16, 16)
    ci = torch.zeros(8, dtype=torch.int32)
    m, w = torch.zeros(4, 32, dtype=torch.bfloat16), torch.ones(32)
    for call in (lambda: cc.ssm_scan_fwd(x, dt, A, B, C), lambda: cc.ssm_scan_bwd(x, x, dt, A, B, C),
                 lambda: cc.ssm_state_update(x, dt, A, B, C, state_pool=pool, cache_indices=ci),
                 lambda: cc.gated_norm_fwd(m, m, w), lambda: cc.gated_norm_bwd(m, m, m, w),
                 lambda: cc.residual_norm_fwd(m, m, w), lambda: cc.residual_norm_bwd(m, None, m, w)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_shapes_and_types_are_checked():
    x, dt, A, B, C = tensors()
    pool, ci = torch.zeros(9, 2, 16, 16), torch.zeros(8, dtype=torch.int32)
    bad = [((x[0], dt, A, B, C), {}, "x, B"), ((x.float(), dt, A, B, C), {}, "x: need dtype"), ((x, dt.half(), A, B, C), {}, "dt"),
           ((x, dt[:4], A, B, C), {}, "dt"), ((x, dt, A[:1], B, C), {}, "A"), ((x, dt, A.double(), B, C), {}, "A"),
           ((x, dt, A, B, C[:, :, :8]), {}, "C"), ((x, dt, A, B.transpose(0, 2), C), {}, "B|divisible|C"),
           ((x.transpose(1, 2).contiguous().transpose(1, 2), dt, A, B, C), {}, "contiguous"),
           ((x, dt, A, B, C), dict(seqlen=3), "seqlen"),
           ((x, dt, A, B, C), dict(cu_seqlens=torch.zeros(3)), "cu_seqlens"),
           ((x, dt, A, B, C), dict(cu_seqlens=ci, seqlen=8), "one of them"),
           ((x, dt, A, B, C), dict(state_pool=pool), "cache_indices"),
           ((x, dt, A, B, C), dict(cache_indices=ci), "state_pool"),
           ((x, dt, A, B, C), dict(state_pool=pool, cache_indices=ci, initial_state=pool), "not together"),
           ((x, dt, A, B, C), dict(state_pool=pool[:, :1], cache_indices=ci), "state_pool"),
           ((x, dt, A, B, C), dict(state_pool=pool, cache_indices=ci.long()), "cache_indices"),
           ((x, dt, A, B, C), dict(initial_state=pool), "1 states|initial_state"),
           ((x, dt, A, B, C), dict(seqlen=4, final_state=pool[:1]), "final_state")]
    for args, kw, word in bad:
        with pytest.raises(ValueError, match=word):
            cc.ssm_scan_fwd(*args, **kw)
    with pytest.raises(ValueError, match="cache_indices"):
        cc.ssm_state_update(x, dt, A, B, C, state_pool=pool, cache_indices=ci[:3])
    m, w = torch.zeros(4, 32, dtype=torch.bfloat16), torch.ones(32)
    for call, word in ((lambda: cc.gated_norm_fwd(m, m[:, :16], w), "gate"), (lambda: cc.gated_norm_fwd(m, m, w[:3]), "weight"),
                       (lambda: cc.gated_norm_fwd(m, m, w, group_size=5), "group_size"),
                       (lambda: cc.gated_norm_fwd(m.t(), m.t(), torch.ones(4)), "contiguous"),
                       (lambda: cc.gated_norm_fwd(m[0], m, w), "2-D"),
                       (lambda: cc.residual_norm_fwd(m, m.half(), w), "residual"),
                       (lambda: cc.residual_norm_bwd(m, m.float(), m, w), "dresidual_out")):
        with pytest.raises(ValueError, match=word):
            call()


def test_reference_gradients_by_differences():
    """The float64 gradient the GPU tests compare with, against central differences of the definition."""
    import ssm_reference as ref
    gen = torch.Generator().manual_seed(3)
    R, H, P, G, N = 7, 4, 3, 2, 5
    t = dict(x=torch.randn(R, H, P, generator=gen), dt=torch.randn(R, H, generator=gen), A=-torch.rand(H, generator=gen) - 0.1,
             B=torch.randn(R, G, N, generator=gen), C=torch.randn(R, G, N, generator=gen), D=torch.randn(H, generator=gen),
             bias=torch.randn(H, generator=gen), S0=torch.randn(2, H, P, N, generator=gen))
    t = {k: v.double() for k, v in t.items()}
    dy, dS = torch.randn(R, H, P, generator=gen).double(), torch.randn(2, H, P, N, generator=gen).double()
    bounds = [(0, 3), (3, 7)]

    def loss(v):
        y, fin, _ = ref.scan(*(v[k] for k in ("x", "dt", "A", "B", "C", "D", "bias")), bounds, v["S0"])
        return float((y * dy).sum() + (fin * dS).sum())

    _, _, g = ref.scan(*(t[k] for k in ("x", "dt", "A", "B", "C", "D", "bias")), bounds, t["S0"], dy=dy, dS=dS)
    for k, name in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"), ("bias", "ddt_bias"), ("S0", "dS0")):
        v = torch.randn(t[k].shape, generator=gen).double()
        e = 1e-6
        slope = (loss({**t, k: t[k] + e * v}) - loss({**t, k: t[k] - e * v})) / (2 * e)
        want = float((g[name] * v).sum())
        assert abs(slope - want) <= 1e-7 * max(1.0, abs(want)) * 10, (k, slope, want)
