"""Refusals of the delta rule's, the layer norm's and the slot copies' entry points, decided on the host (CPU only): the C
ABI's by fake addresses that are compared and never read, the torch binding's by host tensors; and what the binding does
besides calling the library, with a recorder in its place."""
import ctypes
import os
import re

import pytest

from causal_depthwise_conv1d_width_amd import _lib

torch = pytest.importorskip("torch")

import causal_depthwise_conv1d_width_amd as cc  # noqa: E402
from causal_depthwise_conv1d_width_amd import delta  # noqa: E402
from test_ssm_stream import Ops, Recorder  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EWORKSPACE = 0, 1, 2
bf16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from causal_depthwise_conv1d_width_amd.build import build
        build()
    return _lib.load_delta()


def test_header_and_binding_agree(lib):
    text = open(os.path.join(ROOT, "include", "delta.h")).read()
    names = set(re.findall(r"^(?:int|size_t)\s+(\w+)\s*\(", text, re.M))
    assert names == set(_lib.DELTA_SIGNATURES)
    for n in names:
        assert hasattr(lib, n)
    for n, (_, args) in _lib.DELTA_SIGNATURES.items():
        head = re.search(r"^(?:int|size_t) %s\((.*?)\);" % n, text, re.S | re.M).group(1)
        assert head.count(",") + 1 == len(args), n


class Call:
    """Arguments of one entry point at fake, disjoint addresses, changed by name."""

    def __init__(self):
        self.next = 1 << 40

    def at(self, nbytes):
        p = self.next
        self.next += (nbytes + 4096 + 255) // 256 * 256
        return p

    def scan(self, lib, which="fwd", **kw):
        R, H, P, G, N, nseq = kw.get("rows", 100), kw.get("H", 4), kw.get("P", 64), kw.get("G", 2), kw.get("N", 64), 3
        hp, gn, big = H * P, G * N, 1 << 22
        v = dict(gates=1, softplus=1, norm=1, scale=0.125, beta=1.0, eps=1e-6)
        v.update({k: self.at(big) for k in ("dy", "q", "k", "v", "dt", "b", "A", "bias", "y", "S0", "dS", "dq", "dk", "dv", "ddt",
                                            "db", "dA", "dbias", "dS0", "cu", "ci", "hi", "fin")})
        v.update(q_ld=gn, k_ld=gn, v_ld=hp, dt_ld=H, b_ld=H, y_ld=hp, dy_ld=hp, dq_ld=gn, dk_ld=gn, dv_ld=hp, ddt_ld=H, db_ld=H,
                 seq_idx=None, seqlen=0, ws=self.at(1 << 30), ws_bytes=1 << 30, slots=8, s_slot=hp * N)
        v.update({k: (v[x] if isinstance(x, str) else x) for k, x in kw.items()})
        sh = ctypes.byref(_lib.DeltaShape(H, P, G, N, v["gates"], v["softplus"], v["norm"], v["scale"], v["beta"], v["eps"]))
        seq = _lib.Seq(v["cu"], nseq, v["seq_idx"], v["seqlen"])
        q = None if kw.get("no_seq") else ctypes.byref(seq)
        ins = [e for n in ("q", "k", "v", "dt", "b") for e in (v[n], v[n + "_ld"])] + [v["A"], v["bias"]]
        if which == "bwd":
            outs = [e for n in ("dq", "dk", "dv", "ddt", "db") for e in (v[n], v[n + "_ld"])]
            return lib.delta_scan_bwd(sh, R, v["dy"], v["dy_ld"], *ins, q, v["S0"], v["dS"], *outs, v["dA"], v["dbias"], v["dS0"],
                                      v["ws"], v["ws_bytes"], None)
        st = ctypes.byref(_lib.SsmStates(v.get("initial", v["S0"]), v["fin"], v["slots"], v["s_slot"], v["ci"], v["hi"]))
        if which == "step":
            return lib.delta_state_update(sh, R, *ins, None if kw.get("no_pool") else st, v["y"], v["y_ld"], None)
        return lib.delta_scan_fwd(sh, R, *ins, q, st, v["y"], v["y_ld"], v["ws"], v["ws_bytes"], None)


inf, nan = float("inf"), float("nan")
SHARED = [dict(H=0), dict(P=0), dict(G=3), dict(N=0), dict(N=257), dict(rows=-1), dict(gates=2), dict(softplus=2), dict(norm=2),
          dict(scale=inf), dict(scale=nan), dict(beta=0.0), dict(beta=-1.0), dict(beta=inf), dict(beta=nan), dict(eps=-1e-6),
          dict(eps=nan), dict(eps=inf), dict(q_ld=10), dict(k_ld=10), dict(v_ld=10), dict(dt_ld=3), dict(b_ld=3), dict(A=None),
          dict(q=None), dict(k=None), dict(v=None), dict(dt=None), dict(b=None), dict(v=(1 << 40) + 1), dict(b=(1 << 40) + 2),
          dict(q_ld=1 << 60)]
PACKED = [dict(no_seq=True), dict(seq_idx=4096), dict(cu=None, seqlen=0), dict(cu=None, seqlen=33), dict(ws=(1 << 45) + 8),
          dict(v_ld=(1 << 24) + 1), dict(k_ld=1 << 47)]
FWD = [dict(y=None), dict(y_ld=1), dict(y="q"), dict(y="k"), dict(y="v"), dict(y="b"), dict(y="cu"), dict(y="A"), dict(fin="v"),
       dict(fin="y"), dict(ws="q"), dict(ws="S0"), dict(ws="fin"), dict(slots=0), dict(s_slot=5), dict(ci=None, slots=2),
       dict(initial=None, fin=None), dict(y="S0"), dict(y="ci")]
BWD = [dict(dy=None), dict(dq=None), dict(dk=None), dict(dv=None), dict(ddt=None), dict(db=None), dict(dA=None), dict(dy_ld=1),
       dict(dq_ld=1), dict(ddt_ld=1), dict(db_ld=3), dict(dq="dk"), dict(dv="dy"), dict(dv="v"), dict(dk="k"), dict(db="b"),
       dict(ddt="db"), dict(dS0="dS"), dict(dS0="S0"), dict(dA="A"), dict(dbias="cu"), dict(ws="v"), dict(ws="dq")]


@pytest.mark.parametrize("which,kw", [("fwd", kw) for kw in SHARED + PACKED + FWD] + [("bwd", kw) for kw in SHARED + PACKED + BWD],
                         ids=str)
def test_scans_refuse(lib, which, kw):
    assert Call().scan(lib, which, **kw) == EINVAL


@pytest.mark.parametrize("kw", SHARED + [dict(y=None), dict(y_ld=1), dict(ci=None), dict(initial=None), dict(fin="v"), dict(y="q"),
                                         dict(y="ci"), dict(y="S0"), dict(slots=0), dict(s_slot=1), dict(no_pool=True)], ids=str)
def test_step_refuses(lib, kw):
    c = Call()
    base = dict(fin="S0", s_slot=4 * 64 * 64)
    if kw.get("y") == "S0":
        base["y"] = "S0"
    assert c.scan(lib, "step", **{**base, **kw}) == EINVAL


def test_workspaces(lib):
    for which in ("fwd", "bwd"):
        assert Call().scan(lib, which, ws_bytes=0) == EWORKSPACE
        assert Call().scan(lib, which, ws=None) == EWORKSPACE
    sh = _lib.DeltaShape(4, 64, 2, 128, 1, 1, 1, 1.0, 1.0, 0.0)
    bad = _lib.DeltaShape(4, 64, 3, 128, 1, 1, 1, 1.0, 1.0, 0.0)
    for need in (lib.delta_scan_fwd_workspace_bytes, lib.delta_scan_bwd_workspace_bytes):
        assert need(ctypes.byref(bad), 640, 1) == 0 and need(None, 640, 1) == 0
        assert need(ctypes.byref(sh), 640, 1) > 0
        exact = need(ctypes.byref(_lib.DeltaShape(4, 64, 2, 64, 1, 1, 1, 1.0, 1.0, 0.0)), 100, 3)
        assert Call().scan(lib, "bwd" if need is lib.delta_scan_bwd_workspace_bytes else "fwd", ws_bytes=exact - 1) == EWORKSPACE


def test_interleaved_columns_are_not_an_overlap(lib):
    """Column ranges of one wider array may be read and written side by side; shared columns may not."""
    c = Call()
    row = c.at(1 << 24)
    ld = 2 * 64 * 2 + 4 * 64
    side = dict(dq=row, dq_ld=ld, dk=row + 2 * 128, dk_ld=ld, dv=row + 2 * 256, dv_ld=ld)
    assert c.scan(lib, "bwd", ws_bytes=0, **side) == EWORKSPACE
    assert c.scan(lib, "bwd", **dict(side, dk=row + 2 * 127)) == EINVAL
    assert c.scan(lib, "bwd", **dict(side, dv=row + 2 * 255)) == EINVAL


def layer(lib, which, **kw):
    c = Call()
    v = dict(rows=10, d=96, x=c.at(1 << 20), r=c.at(1 << 20), ro=c.at(1 << 20), y=c.at(1 << 20), w=c.at(1 << 16), b=c.at(1 << 16),
             dy=c.at(1 << 20), dr=c.at(1 << 20), h=c.at(1 << 20), dx=c.at(1 << 20), dres=c.at(1 << 20), dw=c.at(1 << 16),
             db=c.at(1 << 16), ws=c.at(1 << 24), ws_bytes=1 << 24, ld=96, wd=1, rt=1, eps=1e-5)
    v.update({k: (v[x] if isinstance(x, str) else x) for k, x in kw.items()})
    R, d, ld = v["rows"], v["d"], v["ld"]
    if which == "fwd":
        return lib.layer_norm_fwd(R, d, v["x"], ld, v["r"], ld, v["rt"], 1.0, v["w"], v["b"], v["wd"], v["eps"], v["y"], ld, v["ro"],
                                  ld, None)
    return lib.layer_norm_bwd(R, d, v["dy"], ld, v["dr"], ld, v["h"], ld, v["rt"], 1.0, v["w"], v["wd"], v["eps"], v["dx"], ld,
                              v["dres"], ld, v["dw"], v["db"], v["ws"], v["ws_bytes"], None)


@pytest.mark.parametrize("which,kw", [(w, kw) for w, own in {
    "fwd": [dict(x=None), dict(y=None), dict(ro=None), dict(rt=2), dict(y="x"), dict(y="r"), dict(y="ro"), dict(ro="x"), dict(y="w"),
            dict(y="b"), dict(ro="b"), dict(b=(1 << 50) + 2), dict(r=(1 << 50) + 2)],
    "bwd": [dict(dy=None), dict(h=None), dict(dx=None), dict(dw=None), dict(rt=2), dict(dx="dy"), dict(dx="h"), dict(dx="dres"),
            dict(dx="dr"), dict(dres="h"), dict(dw="w"), dict(dw="db"), dict(db="dr"), dict(ws="dr"), dict(ws="h"),
            dict(dw=(1 << 50) + 2), dict(ws=(1 << 50) + 8)],
}.items() for kw in own + [dict(rows=-1), dict(d=0), dict(d=32769, ld=32769), dict(w=None), dict(wd=2), dict(ld=95), dict(eps=-1.0),
                           dict(eps=nan), dict(rows=1 << 60)]], ids=str)
def test_layer_norm_refuses(lib, which, kw):
    assert layer(lib, which, **kw) == EINVAL


def test_layer_norm_workspaces(lib):
    assert layer(lib, "bwd", ws_bytes=4) == EWORKSPACE
    assert layer(lib, "bwd", ws=None) == EWORKSPACE
    assert lib.layer_norm_bwd_workspace_bytes(10, 32769) == 0 and lib.layer_norm_bwd_workspace_bytes(10, 100) >= 2 * 100 * 4


def slots(lib, npools=2, n=4, source=1 << 50, target=1 << 51, **kw):
    p = dict(ptr=1 << 40, slots=8, slot_bytes=100, s_slot=128)
    p.update(kw)
    pools = (_lib.SlotPool * 2)(_lib.SlotPool(1 << 45, 8, 64, 64), _lib.SlotPool(p["ptr"], p["slots"], p["slot_bytes"], p["s_slot"]))
    return lib.state_copy(None if kw.get("no_pools") else pools, npools, n, source, target, None)


@pytest.mark.parametrize("kw", [dict(npools=-1), dict(npools=9), dict(n=-1), dict(n=8193), dict(source=None), dict(target=None),
                                dict(source=(1 << 50) + 2), dict(target=(1 << 51) + 1), dict(ptr=None), dict(slots=-1),
                                dict(slot_bytes=-1), dict(s_slot=99), dict(s_slot=1 << 62), dict(ptr=(1 << 45) + 8),
                                dict(source=(1 << 40) + 256), dict(target=(1 << 40) + 256), dict(no_pools=True)], ids=str)
def test_state_copy_refuses(lib, kw):
    kw = dict(kw)
    assert slots(lib, **kw) == EINVAL


# ------------------------------------------------------------------ the torch binding
R, H, P, G, N = 8, 2, 16, 1, 16


def tensors():
    k = torch.zeros(R, G, N, dtype=bf16)
    return k, k.clone(), torch.zeros(R, H, P, dtype=bf16), torch.zeros(R, H), torch.zeros(R, H), torch.zeros(H)


def test_host_tensors_are_refused():
    args = tensors()
    pool, ci = torch.zeros(9, H, P, N), torch.zeros(8, dtype=torch.int32)
    m, w = torch.zeros(4, 32, dtype=bf16), torch.ones(32)
    for call in (lambda: cc.delta_scan_fwd(*args), lambda: cc.delta_scan_bwd(args[2], *args),
                 lambda: cc.delta_state_update(*args, state_pool=pool, cache_indices=ci), lambda: cc.layer_norm_fwd(m, w),
                 lambda: cc.layer_norm_bwd(m, m, w), lambda: cc.state_copy(pool, ci, ci)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_shapes_and_types_are_checked():
    q, k, v, dt, b, A = tensors()
    pool, ci = torch.zeros(9, H, P, N), torch.zeros(8, dtype=torch.int32)
    bad = [((q[0], k, v, dt, b, A), {}, "q, k, v"), ((q.float(), k, v, dt, b, A), {}, "q: need dtype"),
           ((q, k, v, dt.half(), b.half(), A), {}, "dt, b"), ((q, k, v, dt, b.to(bf16), A), {}, "dt, b"),
           ((q, k, v, dt[:4], b, A), {}, "dt"), ((q, k, v, dt, b, A[:1]), {}, "A"), ((q, k, v, dt, b, A.double()), {}, "A"),
           ((q[:, :, :8], k, v, dt, b, A), {}, "q"), ((q, k.expand(R, 3, N), v, dt, b, A), {}, "divisible"),
           ((q, torch.zeros(R, 1, 257, dtype=bf16), v, dt, b, A), {}, "256"),
           ((q, k, v.transpose(1, 2).contiguous().transpose(1, 2), dt, b, A), {}, "contiguous"),
           ((q, k, v, dt, b, A), dict(norm_eps=-1.0), "norm_eps"), ((q, k, v, dt, b, A), dict(norm_eps=nan), "norm_eps"),
           ((q, k, v, dt, b, A), dict(beta_max=0), "beta_max"), ((q, k, v, dt, b, A), dict(beta_max=inf), "beta_max"),
           ((q, k, v, dt, b, A), dict(scale=nan), "scale"), ((q, k, v, dt, b, A), dict(seqlen=3), "seqlen"),
           ((q, k, v, dt, b, A), dict(cu_seqlens=torch.zeros(3)), "cu_seqlens"),
           ((q, k, v, dt, b, A), dict(cu_seqlens=ci, seqlen=8), "one of them"),
           ((q, k, v, dt, b, A), dict(state_pool=pool), "cache_indices"),
           ((q, k, v, dt, b, A), dict(cache_indices=ci), "state_pool"),
           ((q, k, v, dt, b, A), dict(state_pool=pool, cache_indices=ci, initial_state=pool), "not together"),
           ((q, k, v, dt, b, A), dict(state_pool=pool[:, :1], cache_indices=ci), "state_pool"),
           ((q, k, v, dt, b, A), dict(state_pool=pool, cache_indices=ci.long()), "cache_indices"),
           ((q, k, v, dt, b, A), dict(initial_state=pool), "1 states|initial_state"),
           ((q, k, v, dt, b, A), dict(seqlen=4, final_state=pool[:1]), "final_state")]
    for args, kw, word in bad:
        with pytest.raises(ValueError, match=word):
            cc.delta_scan_fwd(*args, **kw)
    with pytest.raises(ValueError, match="cache_indices"):
        cc.delta_state_update(q, k, v, dt, b, A, state_pool=pool, cache_indices=ci[:3])
    with pytest.raises(ValueError, match="required"):
        cc.delta_state_update(q, k, v, dt, b, A, state_pool=pool, cache_indices=None)
    m, w = torch.zeros(4, 32, dtype=bf16), torch.ones(32)
    for call, word in ((lambda: cc.layer_norm_fwd(m[0], w), "2-D"), (lambda: cc.layer_norm_fwd(m, w[:3]), "weight"),
                       (lambda: cc.layer_norm_fwd(m, w, w.to(bf16)), "bias"),
                       (lambda: cc.layer_norm_fwd(m, w, scale=2.0), "need a residual"),
                       (lambda: cc.layer_norm_fwd(m, w, residual_out=m), "need a residual"),
                       (lambda: cc.layer_norm_bwd(m, m, w, dresidual=m), "residual=True")):
        with pytest.raises(ValueError, match=word):
            call()
    for call, word in ((lambda: cc.state_copy([], ci, ci), "1 to 8"), (lambda: cc.state_copy([pool] * 9, ci, ci), "1 to 8"),
                       (lambda: cc.state_copy(pool, ci, ci[:3]), "same length"),
                       (lambda: cc.state_copy(pool, ci.long(), ci), "source"),
                       (lambda: cc.state_copy(pool[:, :, ::2], ci, ci), "without gaps"),
                       (lambda: cc.state_copy(pool[:1].expand(4, H, P, N), ci, ci), "overlap"),
                       (lambda: cc.state_copy(pool, torch.zeros(8193, dtype=torch.int32), torch.zeros(8193, dtype=torch.int32)),
                        "8192")):
        with pytest.raises(ValueError, match=word):
            call()


@pytest.fixture
def recorder(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(_lib, "load_delta", lambda: rec)
    monkeypatch.setattr(delta, "_on", lambda x, *tensors: 0)
    monkeypatch.setattr(delta, "_stream", lambda stream, dev: 0)
    return rec


def calls():
    args = tensors()
    pool, ci, S = torch.zeros(9, H, P, N), torch.zeros(8, dtype=torch.int32), torch.zeros(1, H, P, N)
    m, r, w = torch.zeros(4, 32, dtype=bf16), torch.zeros(4, 32), torch.ones(32)
    return dict(
        scan_fwd=lambda **k: cc.delta_scan_fwd(*args, **k),
        scan_fwd_pool=lambda **k: cc.delta_scan_fwd(*args, seqlen=1, state_pool=pool, cache_indices=ci, **k),
        scan_bwd=lambda **k: cc.delta_scan_bwd(args[2], *args, args[5], initial_state=S, **k),
        step=lambda **k: cc.delta_state_update(*args, state_pool=pool, cache_indices=ci, **k),
        layer_fwd=lambda **k: cc.layer_norm_fwd(m, w, w, residual=r, **k),
        layer_bwd=lambda **k: cc.layer_norm_bwd(m, r, w, residual=True, **k))


@pytest.mark.parametrize("name", list(calls()))
def test_nothing_runs_beside_the_library(recorder, name):
    """New tensors are left as they are allocated: no fill, copy or conversion."""
    call = calls()[name]
    with Ops() as ops:
        call()
    assert set(ops.names) <= {"empty", "new_empty"}, ops.names


def test_missing_flags_stay_missing(recorder):
    calls()["scan_fwd_pool"]()
    assert recorder.states.has_initial_state is None and recorder.states.cache_indices
    assert recorder.states.initial == recorder.states.final


@pytest.mark.parametrize("name", list(calls()))
def test_new_arrays_belong_to_the_stream(recorder, name, monkeypatch):
    """Results and workspaces are allocated on the stream argument, and the current stream's use of the results is
    made known to the allocator."""
    call, side, inside, kept, where = calls()[name], object(), [], [], []

    class On:
        def __init__(self, s):
            assert s is side

        def __enter__(self):
            inside.append(True)

        def __exit__(self, *args):
            inside.pop()

    class Allocations(Ops):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = super().__torch_dispatch__(func, types, args, kwargs)
            if "empty" in self.names[-1]:
                where.append((bool(inside), out.data_ptr()))
            return out

    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append((t.data_ptr(), s)), raising=False)
    with Allocations():
        got = call(stream=side)
    got = [got] if isinstance(got, torch.Tensor) else [t for t in got if t is not None]
    assert where and all(on for on, _ in where)
    assert sorted(kept) == sorted((t.data_ptr(), "current") for t in got)


def test_package_names():
    for name in ("delta_scan_fwd", "delta_scan_bwd", "delta_state_update", "layer_norm_fwd", "layer_norm_bwd", "state_copy",
                 "DeltaGrads", "LayerNormGrads"):
        assert getattr(cc, name) is getattr(delta, name) and name in cc.__all__
