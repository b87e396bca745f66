"""GPU: the delta rule's forward with many walks (64 columns a block) gives the bits of the same sequences one at a time, which
are few enough for 32 columns a block and are tested against float64; and float64 itself for one such call.  Tolerances: as in
test_gpu_delta.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import causal_depthwise_conv1d_width_amd as cc  # noqa: E402
from test_gpu_delta import Problem, bf16, f32  # noqa: E402

CUS = 256
LENS = [70, 0, 1, 130, 63, 64, 5, 65, 200]


def many(lens, H, P):
    return len(lens) * H * ((P + 31) // 32) > CUS >= H * ((P + 31) // 32)


@pytest.mark.parametrize("H,P,G,N", [(30, 40, 2, 64), (30, 33, 3, 37), (30, 64, 1, 128), (16, 128, 2, 72), (24, 100, 4, 128)], ids=str)
@pytest.mark.parametrize("kind", ["norm", "raw", "not finite"])
def test_bits_of_sequences_alone(H, P, G, N, kind):
    assert many(LENS, H, P)
    p = Problem(LENS, H, P, G, N, seed=N, norm=kind != "raw", beta=1.0 if kind == "norm" else 1.5, gates=f32 if kind == "norm" else bf16,
                pad=3, first=2, key=1.0 if kind == "norm" else 0.8, wide=8 if kind == "raw" else 0)
    if kind == "not finite":
        s = p.bounds[3][0]
        p.v[s + 70, 1, 3] = float("inf")
        p.k[s + 100, G - 1, 0] = float("nan")
        p.q[p.bounds[0][0] + 9, 0, 0] = float("-inf")
        p.dt[p.bounds[8][0] + 66, 0] = float("nan")
    slots = torch.tensor([3, 9, 0, 1, -1, 7, 2, 12, 5], dtype=torch.int32, device="cuda")  # 12: past the pool
    flags = torch.tensor([1, 1, 0, 1, 1, 0, 0, 1, 1], dtype=torch.bool, device="cuda")
    start = torch.randn(11, H, P, N, generator=torch.Generator().manual_seed(1)).cuda()
    pool, alone = start.clone(), start.clone()
    y = torch.full((p.R, H, P), 7.0, dtype=bf16, device="cuda")
    cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, state_pool=pool, cache_indices=slots, has_initial_state=flags, out=y, **p.kw)
    for i, (s, e) in enumerate(p.bounds):
        one = torch.full_like(y, 7.0)
        cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu[i:i + 2], state_pool=alone, cache_indices=slots[i:i + 1],
                          has_initial_state=flags[i:i + 1], out=one, **p.kw)
        assert torch.equal(y[s:e].view(torch.int16), one[s:e].view(torch.int16)), i
    assert bool((y[:2] == 7).all()) and bool((y[-3:] == 7).all())
    assert torch.equal(pool.view(torch.int32), alone.view(torch.int32))
    assert bool(torch.isfinite(y[p.bounds[6][0]:p.bounds[6][1]]).all())


def test_against_float64():
    lens = [65, 3, 0, 70]
    p = Problem(lens, 40, 40, 2, 72, seed=4)
    assert many(lens, 40, 40)
    final = torch.full((4, 40, 40, 72), float("nan"), device="cuda")
    y = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, initial_state=p.S0, final_state=final, **p.kw)
    p.check(y, final, p.reference(p.S0))


def test_many_short_sequences():
    """More sequences than a block that orders them has threads, most of them empty or of one row."""
    lens = [i % 3 for i in range(700)] + [140]
    p = Problem(lens, 2, 16, 1, 16, seed=6)
    final = torch.full((len(lens), 2, 16, 16), float("nan"), device="cuda")
    y = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, initial_state=p.S0, final_state=final, **p.kw)
    p.check(y, final, p.reference(p.S0))
    g = cc.delta_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu, initial_state=p.S0, dfinal_state=p.dS, **p.kw)
    for i in (0, 1, 2, 350, 351, 352, 698, 699, 700):
        s, e = p.bounds[i]
        if e > s:
            one = cc.delta_scan_bwd(p.dy, *p.args(), cu_seqlens=p.cu[i:i + 2], initial_state=p.S0[i:i + 1].contiguous(),
                                    dfinal_state=p.dS[i:i + 1].contiguous(), **p.kw)
            # the sign that a walk begins with goes by the sequence's number: the same values to their rounding
            for name in ("dq", "dk", "dv"):
                a, b = getattr(g, name)[s:e].float(), getattr(one, name)[s:e].float()
                assert float((a - b).abs().max()) <= 2.0 ** -7 * float(b.abs().max()), (name, i)
        else:
            assert torch.equal(g.dinitial_state[i], p.dS[i])


def test_rows_whose_squares_pass_fp32():
    """Unit keys do not depend on their length.  The forward brings rows to one size first; the step, which sums the squares
    as they are, gives no number rather than a wrong one."""
    p = Problem([70], 2, 32, 1, 64, seed=8, norm_eps=0.0)
    want = cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, **p.kw)
    p.k.mul_(2.0 ** 70)
    assert bool(torch.isfinite(p.k).all())
    assert torch.equal(cc.delta_scan_fwd(*p.args(), cu_seqlens=p.cu, **p.kw), want)
    pool = torch.zeros(3, 2, 32, 64, device="cuda")
    slots = torch.tensor([1], dtype=torch.int32, device="cuda")
    y = cc.delta_state_update(*(t[:1] for t in p.args()[:5]), p.A, p.bias, state_pool=pool, cache_indices=slots, **p.kw)
    assert bool(torch.isnan(y).all()) and bool(torch.isnan(pool[1]).all()) and float(pool[[0, 2]].abs().max()) == 0
