"""One mixer block on the package's kernels: training forward and backward, prefill and decode.

    (h, r') = residual_norm(x, r)                 residual addition and RMS norm
    [z | xBC | dt] = h W_in                       one projection (a library product)
    [xs | B | C] = silu(conv(xBC))                width-4 causal convolution, packed rows
    y = scan(xs, softplus(dt + bias), A, B, C, D)
    out = gated_norm(y, z) W_out

The column ranges of a projection are passed as they lie (rows with a stride), and the backward pass
writes its gradients into the ranges of one array, so nothing is copied between the kernels.

    python examples/mixer_block.py                trains a block for some steps, then prefills and decodes
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import causal_depthwise_conv1d_width_amd as cc  # noqa: E402

NAMES = ("norm", "w_in", "conv", "conv_bias", "A", "D", "dt_bias", "gate_norm", "w_out")


class MixerBlock:
    """heads x head_dim inner channels; groups of heads share B and C of `state` columns."""

    def __init__(self, d_model, heads, head_dim=64, groups=1, state=128, device="cuda", seed=0):
        self.d, self.H, self.P, self.G, self.N = d_model, heads, head_dim, groups, state
        self.inner, self.conv_dim = heads * head_dim, heads * head_dim + 2 * groups * state
        gen = torch.Generator().manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=gen) * scale).to(device)

        width = self.inner + self.conv_dim + heads
        self.params = {
            "norm": torch.ones(d_model, device=device),
            "w_in": normal(d_model, width, scale=d_model ** -0.5).bfloat16(),
            "conv": normal(self.conv_dim, 4, scale=0.5),
            "conv_bias": torch.zeros(self.conv_dim, device=device),
            "A": -torch.linspace(1, 8, heads).to(device),
            "D": torch.ones(heads, device=device),
            # softplus(dt_bias) from 0.01 to 0.1
            "dt_bias": torch.expm1(torch.linspace(0.01, 0.1, heads).double()).log().float().to(device),
            "gate_norm": torch.ones(self.inner, device=device),
            "w_out": normal(self.inner, d_model, scale=self.inner ** -0.5).bfloat16(),
        }

    def ranges(self, p):
        """z, xBC and dt of the projection's rows."""
        return p[:, :self.inner], p[:, self.inner:self.inner + self.conv_dim], p[:, self.inner + self.conv_dim:]

    def heads(self, c):
        """x [rows, H, P], B and C [rows, G, N] of the convolution's rows."""
        gn = self.G * self.N
        x, B, C = c[:, :self.inner], c[:, self.inner:self.inner + gn], c[:, self.inner + gn:]
        return x.unflatten(1, (self.H, self.P)), B.unflatten(1, (self.G, self.N)), C.unflatten(1, (self.G, self.N))

    def _out(self, y, z):
        w = self.params
        return cc.gated_norm_fwd(y.flatten(1), z, w["gate_norm"], group_size=self.inner // self.G)

    # ---------------------------------------------------------------- training
    def forward(self, x, residual, *, cu_seqlens=None, seqlen=None):
        """(out, new residual, what the backward pass needs)."""
        w = self.params
        h, res = cc.residual_norm_fwd(x, residual, w["norm"])
        p = h @ w["w_in"]
        z, xbc, dt = self.ranges(p)
        seq = dict(cu_seqlens=cu_seqlens, seqlen=seqlen)
        c = cc.conv1d_fwd(xbc, w["conv"], w["conv_bias"], **seq)
        y = cc.ssm_scan_fwd(*self._scan_inputs(c, dt), **seq)
        g = self._out(y, z)
        return g @ w["w_out"], res, (h, res, p, c, y, g, seq)

    def backward(self, dout, dres, saved):
        """(dx, dresidual, {parameter: gradient}); dres: the new residual's gradient, or None."""
        w = self.params
        h, res, p, c, y, g, seq = saved
        z, xbc, dt = self.ranges(p)
        dp, dc = torch.empty_like(p), torch.empty_like(c)
        dz, dxbc, ddt = self.ranges(dp)
        dxs, dB, dC = self.heads(dc)
        grads = {"w_out": g.T @ dout}
        dy, _, grads["gate_norm"] = cc.gated_norm_bwd(dout @ w["w_out"].T, y.flatten(1), z, w["gate_norm"],
                                                      group_size=self.inner // self.G, dgate=dz)
        s = cc.ssm_scan_bwd(dy.view_as(y), *self._scan_inputs(c, dt), **seq, dx=dxs, dB=dB, dC=dC, ddt=ddt)
        grads.update(A=s.dA, D=s.dD, dt_bias=s.ddt_bias)
        _, grads["conv"], grads["conv_bias"], _ = cc.conv1d_bwd(xbc, dc, w["conv"], w["conv_bias"], **seq, dx=dxbc)
        grads["w_in"] = h.T @ dp
        dx, dresidual, grads["norm"] = cc.residual_norm_bwd(dp @ w["w_in"].T, dres, res, w["norm"])
        return dx, dresidual, grads

    def _scan_inputs(self, c, dt):
        w = self.params
        x, B, C = self.heads(c)
        return x, dt, w["A"], B, C, w["D"], w["dt_bias"]

    # ---------------------------------------------------------------- serving
    def caches(self, slots):
        """Convolution and scan states of `slots` sequences."""
        dev = self.params["norm"].device
        return (torch.zeros(slots, self.conv_dim, 3, dtype=torch.bfloat16, device=dev),
                torch.zeros(slots, self.H, self.P, self.N, device=dev))

    def prefill(self, x, residual, caches, cache_indices, cu_seqlens, has_initial_state=None):
        """Packed prompts (or further pieces of them); the slots' states advance in place."""
        w = self.params
        h, res = cc.residual_norm_fwd(x, residual, w["norm"])
        z, xbc, dt = self.ranges(h @ w["w_in"])
        seq = dict(cu_seqlens=cu_seqlens, cache_indices=cache_indices, has_initial_state=has_initial_state)
        c = cc.conv1d_fwd(xbc, w["conv"], w["conv_bias"], conv_state=caches[0], **seq)
        y = cc.ssm_scan_fwd(*self._scan_inputs(c, dt), state_pool=caches[1], **seq)
        return self._out(y, z) @ w["w_out"], res

    def decode(self, x, residual, caches, cache_indices):
        """One token a sequence."""
        w = self.params
        h, res = cc.residual_norm_fwd(x, residual, w["norm"])
        z, xbc, dt = self.ranges(h @ w["w_in"])
        c = cc.conv1d_state_update(xbc, w["conv"], w["conv_bias"], conv_state=caches[0], cache_indices=cache_indices)
        y = cc.ssm_state_update(*self._scan_inputs(c, dt), state_pool=caches[1], cache_indices=cache_indices)
        return self._out(y, z) @ w["w_out"], res


def plain_block(params, x, residual, bounds, heads, head_dim, groups, state):
    """The block's formulas one token at a time, in elementary operations, differentiable: (out, new residual)."""
    w, (H, P, G, N) = params, (heads, head_dim, groups, state)
    inner = H * P
    res = residual + x
    h = res * torch.rsqrt(res.square().mean(1, keepdim=True) + 1e-5) * w["norm"]
    z, xbc, dt = (h @ w["w_in"]).split([inner, inner + 2 * G * N, H], 1)
    dt = F.softplus(dt + w["dt_bias"])
    rows = []
    for s, e in zip(bounds[:-1], bounds[1:]):
        pad = torch.cat([xbc.new_zeros(3, xbc.shape[1]), xbc[s:e]])
        c = F.silu(sum(pad[k:k + e - s] * w["conv"][:, k] for k in range(4)) + w["conv_bias"])
        S = c.new_zeros(H, P, N)
        for t in range(e - s):
            xs, B, C = c[t, :inner].view(H, P), c[t, inner:inner + G * N].view(G, N), c[t, inner + G * N:].view(G, N)
            B, C = B.repeat_interleave(H // G, 0), C.repeat_interleave(H // G, 0)
            d = dt[s + t]
            S = torch.exp(d * w["A"])[:, None, None] * S + (d[:, None] * xs)[:, :, None] * B[:, None]
            rows.append(((S * C[:, None]).sum(2) + w["D"][:, None] * xs).flatten())
    u = (torch.stack(rows) * F.silu(z)).unflatten(1, (G, inner // G))
    u = (u * torch.rsqrt(u.square().mean(2, keepdim=True) + 1e-5)).flatten(1) * w["gate_norm"]
    return u @ w["w_out"], res


def main():
    block = MixerBlock(512, heads=16, groups=2)
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(4 * 1024, 512, generator=gen).bfloat16().cuda()
    residual, target = torch.zeros_like(x, dtype=torch.float32), torch.roll(x, 1, 0).float()
    for step in range(10):
        out, res, saved = block.forward(x, residual, seqlen=1024)
        off = out.float() + res - target
        loss = off.square().mean()
        g = off * (2 / off.numel())
        _, _, grads = block.backward(g.bfloat16(), g, saved)
        for name, grad in grads.items():
            p = block.params[name]
            p.copy_((p.float() - 30 * grad.float()).to(p.dtype))
        print(f"step {step}: loss {loss.item():.4f}", flush=True)

    lens, slots = [700, 33, 1, 260], torch.tensor([5, 0, 3, 2], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    caches = block.caches(8)
    n = sum(lens)
    out, res = block.prefill(x[:n], residual[:n], caches, slots, cu)
    token = out[cu[1:].long() - 1]
    graph, zero = torch.cuda.CUDAGraph(), torch.zeros_like(token, dtype=torch.float32)
    block.decode(token, zero, block.caches(8), slots)  # the first call of a shape may load kernels
    with torch.cuda.graph(graph):
        nxt, _ = block.decode(token, zero, caches, slots)
    for _ in range(16):
        graph.replay()
        token.copy_(nxt)
    torch.cuda.synchronize()
    print("decoded 16 tokens of 4 sequences, rms", [f"{v:.3f}" for v in token.float().square().mean(1).sqrt().tolist()])


if __name__ == "__main__":
    main()
