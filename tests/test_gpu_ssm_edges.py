"""GPU: the scan where it went wrong once: bits of calls in many pieces, calls on a stream of their own.

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
