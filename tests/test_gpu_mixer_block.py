"""GPU: the example's mixer block against its formulas one token at a time in float64 (plain_block).

Tolerances count roundings along the block, 2^-8 at most each, relative in the 2-norm.  Outputs: the first
norm, the projection, the convolution, three in the scan (state operand, decayed scores, y), the gated
norm, the output: eight, 2^-5.  Gradients see the forward's and as many again on the way back: 2^-4.  The
inputs and weights are the same values on both sides.
"""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))

import mixer_block as mb  # noqa: E402

OUT, GRAD = 2.0 ** -5, 2.0 ** -4


def off(got, want):
    got, want = got.detach().cpu().double(), want.detach().double()
    return float((got - want).norm() / want.norm())


def inputs(n, d, seed=3):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(n, d, generator=gen).bfloat16(), torch.randn(n, d, generator=gen)


@pytest.mark.parametrize("heads,head_dim,groups,state", [(4, 32, 2, 40), (2, 64, 1, 128)])
def test_training_step(heads, head_dim, groups, state):
    lens = [70, 1, 0, 66]
    bounds = [0]
    for n in lens:
        bounds.append(bounds[-1] + n)
    block = mb.MixerBlock(96, heads, head_dim, groups, state)
    x, r = inputs(bounds[-1], 96)
    dout, dres = inputs(bounds[-1], 96, seed=4)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    out, res, saved = block.forward(x.cuda(), r.cuda(), cu_seqlens=cu)
    dx, dr, grads = block.backward(dout.cuda(), dres.cuda(), saved)

    params = {k: v.cpu().double().requires_grad_() for k, v in block.params.items()}
    xd, rd = x.double().requires_grad_(), r.double().requires_grad_()
    want, want_res = mb.plain_block(params, xd, rd, bounds, heads, head_dim, groups, state)
    ((want * dout.double()).sum() + (want_res * dres.double()).sum()).backward()
    assert off(out, want) <= OUT
    assert off(res, want_res) <= 2.0 ** -23
    assert off(dx, xd.grad) <= GRAD
    assert off(dr, rd.grad) <= GRAD
    assert set(grads) == set(mb.NAMES)
    for name in mb.NAMES:
        assert off(grads[name], params[name].grad) <= GRAD, name


def test_prefill_in_pieces_then_decode():
    block = mb.MixerBlock(96, 4, 32, 2, 40)
    lens, first, steps = [90, 7, 131], [64, 3, 50], 4  # the last `steps` tokens are decoded
    bounds = [0]
    for n in lens:
        bounds.append(bounds[-1] + n)
    x, r = inputs(bounds[-1], 96)
    params = {k: v.cpu().double() for k, v in block.params.items()}
    want, _ = mb.plain_block(params, x.double(), r.double(), bounds, 4, 32, 2, 40)

    slots = torch.tensor([4, 1, 2], dtype=torch.int32, device="cuda")
    caches = block.caches(6)
    got = torch.empty(bounds[-1], 96, dtype=torch.float64)
    for lo, hi in ([0, 0, 0], first), (first, [n - steps for n in lens]):
        at = torch.cat([torch.arange(b + s, b + e) for b, s, e in zip(bounds, lo, hi)])
        cu = torch.tensor([0] + [e - s for s, e in zip(lo, hi)]).cumsum(0).int().cuda()
        has = torch.tensor([s > 0 for s in lo], device="cuda")
        out, _ = block.prefill(x[at].cuda(), r[at].cuda(), caches, slots, cu, has)
        got[at] = out.cpu().double()
    for k in range(steps):
        at = torch.tensor([b + n - steps + k for b, n in zip(bounds, lens)])
        out, _ = block.decode(x[at].cuda(), r[at].cuda(), caches, slots)
        got[at] = out.cpu().double()
    assert off(got, want) <= OUT
    assert float(caches[0][[0, 3, 5]].abs().max()) == 0 and float(caches[1][[0, 3, 5]].abs().max()) == 0
