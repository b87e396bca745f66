"""What the torch binding of the scan, step and norms does besides calling the library (CPU only: the library is
a recorder, the tensors are host tensors).  The kernels run on the `stream` argument; work that the binding
itself put on the current stream would not be ordered with them."""
import pytest

from causal_depthwise_conv1d_width_amd import _lib

torch = pytest.importorskip("torch")

from torch.utils._python_dispatch import TorchDispatchMode  # noqa: E402

import causal_depthwise_conv1d_width_amd as cc  # noqa: E402
from causal_depthwise_conv1d_width_amd import ssm  # noqa: E402

bf16 = torch.bfloat16


class Recorder:
    """Every entry point succeeds; workspaces are 64 bytes; the states argument of the last call is kept."""

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return lambda *args: 64

        def call(*args):
            for a in args:
                if isinstance(getattr(a, "_obj", None), _lib.SsmStates):
                    self.states = a._obj
            return _lib.OK
        return call


class Ops(TorchDispatchMode):
    """Names of the torch operations that run."""

    def __enter__(self):
        self.names = []
        return super().__enter__()

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.names.append(func.overloadpacket.__name__)
        return func(*args, **(kwargs or {}))


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(_lib, "load_ssm", lambda: rec)
    monkeypatch.setattr(ssm, "_on", lambda x, *tensors: 0)
    monkeypatch.setattr(ssm, "_stream", lambda stream, dev: 0)
    return rec


R, H, P, G, N = 8, 2, 16, 1, 16


def calls():
    x, B, C = torch.zeros(R, H, P, dtype=bf16), torch.zeros(R, G, N, dtype=bf16), torch.zeros(R, G, N, dtype=bf16)
    scan = (x, torch.zeros(R, H), torch.zeros(H), B, C, torch.zeros(H), torch.zeros(H))
    pool, ci, S = torch.zeros(9, H, P, N), torch.zeros(8, dtype=torch.int32), torch.zeros(1, H, P, N)
    m, r, w = torch.zeros(4, 32, dtype=bf16), torch.zeros(4, 32), torch.ones(32)
    return dict(
        scan_fwd=lambda **k: cc.ssm_scan_fwd(*scan, **k),
        scan_fwd_pool=lambda **k: cc.ssm_scan_fwd(*scan, seqlen=1, state_pool=pool, cache_indices=ci, **k),
        scan_bwd=lambda **k: cc.ssm_scan_bwd(x, *scan, initial_state=S, **k),
        step=lambda **k: cc.ssm_state_update(*scan, state_pool=pool, cache_indices=ci, **k),
        gated_fwd=lambda **k: cc.gated_norm_fwd(m, m, w, **k),
        gated_bwd=lambda **k: cc.gated_norm_bwd(m, m, m, w, **k),
        residual_fwd=lambda **k: cc.residual_norm_fwd(m, r, w, **k),
        residual_bwd=lambda **k: cc.residual_norm_bwd(m, r, r, w, **k))


@pytest.mark.parametrize("name", list(calls()))
def test_nothing_runs_beside_the_library(lib, name):
    """New tensors are left as they are allocated: no fill, copy or conversion."""
    call = calls()[name]
    with Ops() as ops:
        call()
    assert set(ops.names) <= {"empty", "new_empty"}, ops.names


def test_missing_flags_stay_missing(lib):
    calls()["scan_fwd_pool"]()
    assert lib.states.has_initial_state is None and lib.states.cache_indices
    assert lib.states.initial == lib.states.final


@pytest.mark.parametrize("name", list(calls()))
def test_new_arrays_belong_to_the_stream(lib, name, monkeypatch):
    """Results and workspaces are allocated on the stream argument, and the current stream's use of the results is
    made known to the allocator."""
    call, side, inside, kept = calls()[name], object(), [], []

    class On:
        def __init__(self, s):
            assert s is side

        def __enter__(self):
            inside.append(True)

        def __exit__(self, *args):
            inside.pop()

    where = []

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


@pytest.mark.parametrize("name", ["scan_fwd", "scan_bwd", "gated_bwd", "residual_bwd"])
def test_a_workspace_that_repeats_its_bytes_is_refused(lib, name):
    """An expanded tensor counts more bytes than it has, and kernels would write past them."""
    byte = torch.zeros(1, dtype=torch.uint8)
    calls()[name](workspace=byte.repeat(64))
    for ws in (byte.expand(64), torch.zeros(128, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            calls()[name](workspace=ws)
