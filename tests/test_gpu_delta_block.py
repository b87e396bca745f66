"""GPU: a block of the delta rule's operators as they are used together, against its formulas in float64: layer norm of the
residual's sum, projection, convolution, rule, gated norm, projection; trained, prefilled in pieces, forked and swapped
between slots, decoded.

Tolerances count roundings along the block, 2^-8 at most each, relative in the 2-norm.  Three lie before the rule (norm,
projection, convolution) and enter y by q, v and twice by k, which makes twelve; y, the gated norm and the output are three more.
Roundings are independent and add as squares: sqrt(15) 2^-8 < 2^-6, twice that for what products of the rule amplify:
2^-5.  Gradients see the forward's and as many again on the way back: 2^-4.  Inputs and weights are the same values on both
sides.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import torch.nn.functional as F  # noqa: E402

import causal_depthwise_conv1d_width_amd as cc  # noqa: E402
from delta_reference import rule  # noqa: E402

OUT, GRAD = 2.0 ** -5, 2.0 ** -4
D = 96


class Block:
    def __init__(self, H, P, G, N, seed=0):
        self.H, self.P, self.G, self.N = H, P, G, N
        self.inner, self.conv = H * P, H * P + 2 * G * N
        gen = torch.Generator().manual_seed(seed)
        normal = lambda *s, scale: torch.randn(s, generator=gen) * scale  # noqa: E731
        width = self.inner + self.conv + 2 * H
        self.params = {k: v.cuda() for k, v in dict(
            norm=1 + normal(D, scale=0.1), norm_bias=normal(D, scale=0.1), w_in=normal(D, width, scale=D ** -0.5).bfloat16(),
            conv=normal(self.conv, 4, scale=0.5), conv_bias=normal(self.conv, scale=0.1), A=-torch.linspace(1, 4, H),
            dt_bias=torch.linspace(-3, -1, H), gate=1 + normal(self.inner, scale=0.1),
            w_out=normal(self.inner, D, scale=self.inner ** -0.5).bfloat16()).items()}

    def ranges(self, p):
        """z, the convolution's channels, dt and b of the projection's rows."""
        return p.split([self.inner, self.conv, self.H, self.H], 1)

    def heads(self, c):
        gn = self.G * self.N
        q, k, v = c.split([gn, gn, self.inner], 1)
        return q.unflatten(1, (self.G, self.N)), k.unflatten(1, (self.G, self.N)), v.unflatten(1, (self.H, self.P))

    def rest(self, dt, b):
        return dt, b, self.params["A"], self.params["dt_bias"]

    def forward(self, x, r, caches=None, **seq):
        """(out, new residual, saved): with caches, the slots' states advance; without `cu_seqlens`, one token a sequence."""
        w = self.params
        h, res = cc.layer_norm_fwd(x, w["norm"], w["norm_bias"], residual=r)
        z, xc, dt, b = self.ranges(p := h @ w["w_in"])
        if caches is None:
            c = cc.conv1d_fwd(xc, w["conv"], w["conv_bias"], **seq)
            y = cc.delta_scan_fwd(*self.heads(c), *self.rest(dt, b), **seq)
        elif "cu_seqlens" in seq:
            c = cc.conv1d_fwd(xc, w["conv"], w["conv_bias"], conv_state=caches[0], **seq)
            y = cc.delta_scan_fwd(*self.heads(c), *self.rest(dt, b), state_pool=caches[1], **seq)
        else:
            c = cc.conv1d_state_update(xc, w["conv"], w["conv_bias"], conv_state=caches[0], **seq)
            y = cc.delta_state_update(*self.heads(c), *self.rest(dt, b), state_pool=caches[1], **seq)
        g = cc.gated_norm_fwd(y.flatten(1), z, w["gate"], group_size=self.P)
        return g @ w["w_out"], res, (h, res, p, c, y, g, seq)

    def backward(self, dout, dres, saved):
        w = self.params
        h, res, p, c, y, g, seq = saved
        z, xc, dt, b = self.ranges(p)
        dp, dc = torch.full_like(p, float("nan")), torch.full_like(c, float("nan"))
        dz, dxc, ddt, db = self.ranges(dp)
        dq, dk, dv = self.heads(dc)
        grads = {"w_out": g.T @ dout}
        dy, _, grads["gate"] = cc.gated_norm_bwd(dout @ w["w_out"].T, y.flatten(1), z, w["gate"], group_size=self.P, dgate=dz)
        s = cc.delta_scan_bwd(dy.view_as(y), *self.heads(c), *self.rest(dt, b), **seq, dq=dq, dk=dk, dv=dv, ddt=ddt, db=db)
        grads.update(A=s.dA, dt_bias=s.ddt_bias)
        _, grads["conv"], grads["conv_bias"], _ = cc.conv1d_bwd(xc, dc, w["conv"], w["conv_bias"], **seq, dx=dxc)
        grads["w_in"] = h.T @ dp
        n = cc.layer_norm_bwd(dp @ w["w_in"].T, res, w["norm"], residual=True, dresidual_out=dres)
        grads.update(norm=n.dweight, norm_bias=n.dbias)
        return n.dx, n.dresidual, grads

    def caches(self, slots):
        return (torch.zeros(slots, self.conv, 3, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(slots, self.H, self.P, self.N, device="cuda"))

    def plain(self, w, x, r, bounds):
        res = r + x
        h = F.layer_norm(res, (D,), w["norm"], w["norm_bias"])
        z, xc, dt, b = self.ranges(h @ w["w_in"])
        rows = []
        for s, e in zip(bounds[:-1], bounds[1:]):
            pad = torch.cat([xc.new_zeros(3, self.conv), xc[s:e]])
            rows.append(F.silu(sum(pad[k:k + e - s] * w["conv"][:, k] for k in range(4)) + w["conv_bias"]))
        S0 = xc.new_zeros(len(bounds) - 1, self.H, self.P, self.N)
        y, _, _ = rule(*self.heads(torch.cat(rows)), dt, b, w["A"], w["dt_bias"], list(zip(bounds[:-1], bounds[1:])), S0)
        u = (y.flatten(1) * F.silu(z)).unflatten(1, (self.H, self.P))
        u = (u * torch.rsqrt(u.square().mean(2, keepdim=True) + 1e-5)).flatten(1) * w["gate"]
        return u @ w["w_out"], res


def off(got, want):
    got, want = got.detach().cpu().double(), want.detach().double()
    return float((got - want).norm() / want.norm())


def ends(lens):
    return [0] + torch.tensor(lens).cumsum(0).tolist()


def inputs(n, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(n, D, generator=gen).bfloat16(), torch.randn(n, D, generator=gen)


@pytest.mark.parametrize("H,P,G,N", [(4, 32, 2, 40), (2, 64, 1, 128), (3, 20, 3, 136)])
def test_training_step(H, P, G, N):
    bounds = ends([70, 1, 0, 66])
    block = Block(H, P, G, N)
    x, r = inputs(bounds[-1], 3)
    dout, dres = inputs(bounds[-1], 4)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    out, res, saved = block.forward(x.cuda(), r.cuda(), cu_seqlens=cu)
    dx, dr, grads = block.backward(dout.cuda(), dres.cuda(), saved)
    w = {k: v.cpu().double().requires_grad_() for k, v in block.params.items()}
    xd, rd = x.double().requires_grad_(), r.double().requires_grad_()
    want, want_res = block.plain(w, xd, rd, bounds)
    ((want * dout.double()).sum() + (want_res * dres.double()).sum()).backward()
    assert off(out, want) <= OUT
    assert off(res, want_res) <= 2.0 ** -23
    assert off(dx, xd.grad) <= GRAD
    assert off(dr, rd.grad) <= GRAD
    assert set(grads) == set(w)
    for name in w:
        assert off(grads[name], w[name].grad) <= GRAD, name


def test_prefill_fork_swap_decode():
    """Prompts in two pieces into slots; one is forked, two change places; then all are decoded, eagerly and replayed."""
    block = Block(4, 32, 2, 40)
    lens, first, steps = [90, 7, 131], [64, 3, 50], 4
    old = ends(lens)
    # after the copies, request i runs in slots[i]; request 3 is a fork of 0
    before, slots = [4, 1, 2], [1, 4, 2, 5]
    parent = [0, 1, 2, 0]
    x, r = inputs(old[-1] + 4 * steps, 5)
    tails = [list(range(old[-1] + steps * i, old[-1] + steps * (i + 1))) for i in range(4)]
    rows = [list(range(old[p], old[p + 1])) + tails[i] for i, p in enumerate(parent)]
    at = [t for seq in rows for t in seq]
    w = {k: v.cpu().double() for k, v in block.params.items()}
    want, _ = block.plain(w, x.double()[at], r.double()[at], ends([len(s) for s in rows]))
    want = dict(zip([(i, t) for i, seq in enumerate(rows) for t in seq], want))

    caches = block.caches(6)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    got = {}
    for lo, hi in ([0, 0, 0], first), (first, lens):
        pick = [t for b, s, e in zip(old, lo, hi) for t in range(b + s, b + e)]
        out, _, _ = block.forward(x[pick].cuda(), r[pick].cuda(), caches, cu_seqlens=ints(ends([e - s for s, e in zip(lo, hi)])),
                                  cache_indices=ints(before), has_initial_state=torch.tensor([s > 0 for s in lo], device="cuda"))
        got.update(zip(pick, out.cpu().double()))
    for i, p in enumerate(parent[:3]):
        for t in rows[i][:lens[p]]:
            assert off(got[t], want[i, t]) <= 2 * OUT  # rows one by one
    assert off(torch.stack([got[t] for t in rows[2][:131]]), torch.stack([want[2, t] for t in rows[2][:131]])) <= OUT
    cc.state_copy(caches, ints([4, 1, 4, 9, -1]), ints([1, 4, 5, 0, 3]))
    assert float(caches[1][[0, 3]].abs().max()) == 0
    saved = [c.clone() for c in caches]

    xs, rs, idx = torch.empty(4, D, dtype=torch.bfloat16, device="cuda"), torch.empty(4, D, device="cuda"), ints(slots)
    eager = []
    for k in range(steps):
        pick = [tails[i][k] for i in range(4)]
        xs.copy_(x[pick]), rs.copy_(r[pick])
        out, _, _ = block.forward(xs, rs, caches, cache_indices=idx)
        eager.append(out.clone())
        assert off(out, torch.stack([want[i, t] for i, t in enumerate(pick)])) <= OUT, k
    assert float(caches[1][[0, 3]].abs().max()) == 0

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _, _ = block.forward(xs, rs, caches, cache_indices=idx)
    for c, s in zip(caches, saved):
        c.copy_(s)
    for k in range(steps):
        pick = [tails[i][k] for i in range(4)]
        xs.copy_(x[pick]), rs.copy_(r[pick])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[k]), k


def test_two_streams_at_once():
    """The same training step on two streams side by side, each with its own workspaces: the bits of one alone."""
    block = Block(2, 64, 1, 128)
    bounds = ends([130, 64, 5, 200])
    x, r = (t.cuda() for t in inputs(bounds[-1], 7))
    dout, dres = (t.cuda() for t in inputs(bounds[-1], 8))
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")

    def step():
        out, res, saved = block.forward(x, r, cu_seqlens=cu)
        dx, dr, grads = block.backward(dout, dres, saved)
        return [out, res, dx, dr, grads["A"], grads["dt_bias"], grads["norm"], grads["norm_bias"]]

    alone = step()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(step())
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, alone):
            assert torch.equal(a, b)
