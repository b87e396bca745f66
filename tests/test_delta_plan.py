"""The delta rule's workspace plans and the slot copies' grids (CPU only): delta_api.cpp built with g++ against launch stubs
that keep their arguments.  Every array a launch writes has a place of its own inside the workspace."""
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
    out = str(tmp_path_factory.mktemp("plan") / "libdelta_plan.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
                    f"-I{ROOT}/include", f"-I{CSRC}", os.path.join(CSRC, "delta_api.cpp"),
                    os.path.join(TESTS, "delta_stub_launch.cpp"), "-o", out], check=True, capture_output=True)
    lib = ctypes.CDLL(out)
    for name, (res, args) in _lib.DELTA_SIGNATURES.items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib


NAMES = ("keys", "rec", "order", "rec_rev", "tiles", "head")


def call(lib, rows, nseq, H, P, G, N, batch, bwd):
    """Code, workspace bytes and address of a call at fake, disjoint addresses with exactly the workspace asked for."""
    sh = _lib.DeltaShape(H, P, G, N, 1, 1, 1, 1.0, 1.0, 1e-6)
    need = lib.delta_scan_bwd_workspace_bytes if bwd else lib.delta_scan_fwd_workspace_bytes
    ws_bytes = need(ctypes.byref(sh), rows, nseq)
    at = iter(range(1 << 41, 1 << 47, 1 << 41))
    hp, gn = H * P, G * N
    seq = _lib.Seq(None, 0, None, rows // nseq) if batch else _lib.Seq(next(at), nseq, None, 0)
    n = lambda ld: (next(at), ld)  # noqa: E731
    head = (*n(gn), *n(gn), *n(hp), *n(H), *n(H), next(at), next(at), ctypes.byref(seq))
    ws = 1 << 46
    if bwd:
        code = lib.delta_scan_bwd(ctypes.byref(sh), rows, *n(hp), *head, next(at), next(at), *n(gn), *n(gn), *n(hp), *n(H), *n(H),
                                  next(at), next(at), next(at), ws, ws_bytes, None)
    else:
        st = _lib.SsmStates(next(at), next(at), nseq, hp * N, None, None)
        code = lib.delta_scan_fwd(ctypes.byref(sh), rows, *head, ctypes.byref(st), *n(hp), ws, ws_bytes, None)
    return code, ws_bytes, ws


@pytest.mark.parametrize("rows,nseq,H,P,G,N,batch", [
    (1500, 1, 2, 64, 1, 64, False), (2777, 9, 24, 64, 2, 72, False), (2200, 2, 2, 40, 1, 200, True), (1, 1, 1, 1, 1, 1, False),
    (16384, 4, 64, 128, 4, 128, True), (70, 30, 4, 100, 4, 30, False), (64, 1, 3, 65, 3, 256, False)])
@pytest.mark.parametrize("bwd", [False, True])
def test_arrays_are_apart(lib, rows, nseq, H, P, G, N, batch, bwd):
    code, ws_bytes, ws = call(lib, rows, nseq, H, P, G, N, batch, bwd)
    assert code == _lib.OK
    v = (ctypes.c_int64 * 13)()
    lib.delta_last_plan(v)
    # a chunk id for every chunk of any sequences: the rows' own 64-row grid, and a first chunk a sequence
    assert v[12] >= (rows + 63) // 64 + nseq
    used = NAMES if bwd else NAMES[:3]
    need = {k: (v[i] - ws, v[6 + i]) for i, k in enumerate(used) if v[i]}
    assert ("order" in need) == (not batch and nseq > 1)
    end, last = 0, None
    for name, (at, n) in sorted(need.items(), key=lambda e: e[1][0]):
        assert at >= end, f"{name} begins inside {last}"
        assert at % 16 == 0, name
        end, last = at + n, name
    assert end <= ws_bytes, f"{last} ends past the workspace"


def test_sizes_past_64_bits_are_refused(lib):
    for rows, nseq, H, P in ((1 << 40, 1, 1 << 20, 1 << 20), (1 << 50, 1, 64, 64), (1 << 44, 1, 1 << 12, 64)):
        sh = _lib.DeltaShape(H, P, 1, 128, 1, 1, 1, 1.0, 1.0, 1e-6)
        for need in (lib.delta_scan_fwd_workspace_bytes, lib.delta_scan_bwd_workspace_bytes):
            assert need(ctypes.byref(sh), rows, nseq) == 0


def test_more_blocks_than_a_launch_holds_are_refused(lib):
    code, ws_bytes, _ = call(lib, 1 << 20, 1 << 20, 1 << 12, 8, 1, 16, True, False)
    assert code == 1 and ws_bytes > 0


@pytest.mark.parametrize("n", [1, 2, 3, 63, 64, 65, 128, 129, 1000, 8192])
def test_slot_strips_cover_every_byte_once(lib, n):
    sizes = [1, 15, 16, 17, 1 << 20, (1 << 16) + 3]
    pools = (_lib.SlotPool * len(sizes))(*(_lib.SlotPool((1 + i) << 40, 10000, s, s + 5) for i, s in enumerate(sizes)))
    assert lib.state_copy(pools, len(sizes), n, 1 << 44, 1 << 45, None) == _lib.OK
    assert lib.delta_slots_cover() == 1


def test_nothing_to_do_starts_nothing(lib):
    before = lib.delta_launches()
    sh = _lib.DeltaShape(2, 16, 1, 16, 1, 1, 1, 1.0, 1.0, 1e-6)
    seq = _lib.Seq(1 << 40, 0, None, 0)
    rows = (None, 32) * 5
    assert lib.delta_scan_fwd(ctypes.byref(sh), 0, *rows, 1 << 41, None, ctypes.byref(seq), None, None, 32, None, 0, None) == _lib.OK
    pool = _lib.SsmStates(1 << 42, 1 << 42, 4, 512, 1 << 43, None)
    assert lib.delta_state_update(ctypes.byref(sh), 0, *rows, 1 << 41, None, ctypes.byref(pool), None, 32, None) == _lib.OK
    assert lib.layer_norm_fwd(0, 8, None, 8, None, 8, 1, 1.0, 1 << 41, None, 0, 1e-5, None, 8, None, 8, None) == _lib.OK
    assert lib.state_copy(None, 0, 3, 1 << 41, 1 << 42, None) == _lib.OK
    assert lib.state_copy((_lib.SlotPool * 1)(_lib.SlotPool(1 << 40, 4, 64, 64)), 1, 0, None, None, None) == _lib.OK
    assert lib.delta_launches() == before
