"""The scan's workspace plans (CPU only): ssm_api.cpp built with g++ against launch stubs that keep their
arguments.  Every array a launch writes has a place of its own inside the workspace; the two state walks of
the backward, which run in one launch, share none."""
import ctypes
import os
import subprocess

import pytest

from causal_depthwise_conv1d_width_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = os.path.join(ROOT, "tests")
CSRC = os.path.join(ROOT, "causal_depthwise_conv1d_width_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")

pytestmark = pytest.mark.skipif(not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")),
                                reason="HIP headers not installed")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("plan") / "libssm_plan.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
                    f"-I{ROOT}/include", f"-I{CSRC}", os.path.join(CSRC, "ssm_api.cpp"),
                    os.path.join(TESTS, "ssm_stub_launch.cpp"), "-o", out], check=True, capture_output=True)
    lib = ctypes.CDLL(out)
    for name, (res, args) in _lib.SSM_SIGNATURES.items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib


def plan(lib, rows, nseq, H, P, G, N, batch):
    """Workspace arrays (offset, bytes) of a backward call at fake addresses, the workspace's size, rows a piece (log2)."""
    sh = _lib.SsmShape(H, P, G, N, 1, 1)
    ws_bytes = lib.ssm_scan_bwd_workspace_bytes(ctypes.byref(sh), rows, nseq)
    at = iter(range(1 << 41, 1 << 47, 1 << 41))
    p = {k: next(at) for k in ("dy", "x", "dt", "A", "B", "C", "D", "db", "S0", "dS", "dx", "ddt", "dA", "dB", "dC", "dD",
                               "dbias", "dS0", "cu", "ws")}
    hp, gn = H * P, G * N
    seq = _lib.Seq(None, 0, None, rows // nseq) if batch else _lib.Seq(p["cu"], nseq, None, 0)
    code = lib.ssm_scan_bwd(ctypes.byref(sh), rows, p["dy"], hp, p["x"], hp, p["dt"], H, p["A"], p["B"], gn, p["C"], gn,
                            p["D"], p["db"], ctypes.byref(seq), p["S0"], p["dS"], p["dx"], hp, p["ddt"], H, p["dA"], p["dB"],
                            gn, p["dC"], gn, p["dD"], p["dbias"], p["dS0"], p["ws"], ws_bytes, None)
    assert code == _lib.OK
    v = (ctypes.c_int64 * 12)()
    lib.ssm_last_plan(v)
    seg, items, ids, hsplit = v[8:]
    tile = 64 * (64 if N <= 64 else 128 if N <= 128 else 256) * 4
    hpt = H * ((P + 63) // 64)
    need = dict(cs=(v[4], ids * hpt * tile), ct=(v[5], ids * hpt * tile), head=(v[6], ids * H * 12))
    if seg:
        need.update(piece=(v[0], items * hpt * tile), decay=(v[1], items * H * 4), piece_t=(v[2], items * hpt * tile),
                    decay_t=(v[3], items * H * 4))
    if hsplit > 1:
        need["bc"] = (v[7], 2 * hsplit * rows * gn * 4)
    return {k: (a - p["ws"], n) for k, (a, n) in need.items()}, ws_bytes, seg


@pytest.mark.parametrize("rows,nseq,H,P,G,N,batch", [
    (1500, 1, 2, 64, 1, 64, False), (2777, 9, 24, 64, 2, 72, False), (2200, 2, 2, 40, 1, 200, True),
    (16384, 1, 64, 64, 4, 128, True), (16384, 4, 64, 64, 4, 128, True), (70, 3, 4, 100, 4, 30, False)])
def test_backward_arrays_are_apart(lib, rows, nseq, H, P, G, N, batch):
    need, ws_bytes, seg = plan(lib, rows, nseq, H, P, G, N, batch)
    end, last = 0, None
    for name, (at, n) in sorted(need.items(), key=lambda e: e[1][0]):
        assert at >= end, f"{name} begins inside {last}"
        assert at % 16 == 0, name
        end, last = at + n, name
    assert end <= ws_bytes, f"{last} ends past the workspace"
    if rows // nseq >= 1024 and nseq < 4:
        assert 1 << seg <= rows // nseq // 3, "sequences with pieces between the first and the last"
