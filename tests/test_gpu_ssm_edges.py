"""GPU: the scan where it went wrong once: bits of calls in many pieces.

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
