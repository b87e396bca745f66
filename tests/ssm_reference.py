"""The scan, its gradient and the norms in float64 from their definitions, one row at a time (CPU).

Every function also runs on absolute values (``magnitudes=True``): each output is then the sum of its
terms' magnitudes, the scale that rounding errors of the terms are measured against.
"""
import torch


def softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def _heads(t, H):
    return t.repeat_interleave(H // t.shape[0], 0)


def scan(x, dt, A, B, C, D, bias, bounds, S0, *, sp=True, magnitudes=False, dy=None, dS=None):
    """bounds: [(first row, end row)] of the sequences; S0: [nseq, H, P, N].  Returns y, final states and,
    with dy, a dict of gradients (dS: gradient of the final states or None)."""
    f = (lambda t: t.double().abs()) if magnitudes else (lambda t: t.double())
    x, B, C, D, S0 = f(x), f(B), f(C), f(D), f(S0)
    R, H, P = x.shape
    raw = dt.double() + bias.double()
    d = softplus(raw) if sp else raw
    a = torch.exp(d * A.double())
    dm = d.abs() if magnitudes else d
    y = torch.zeros_like(x)
    finals = S0.clone()
    g = None
    if dy is not None:
        dy = f(dy)
        g = dict(dx=torch.zeros_like(x), ddt=torch.zeros_like(raw), dB=torch.zeros_like(B), dC=torch.zeros_like(C),
                 dA=torch.zeros_like(A, dtype=torch.float64), ddt_bias=torch.zeros_like(A, dtype=torch.float64),
                 dS0=torch.zeros_like(S0), dD=torch.zeros_like(D))
        Av = f(A)
    for i, (s, e) in enumerate(bounds):
        S = S0[i].clone()
        kept = [S]
        for t in range(s, e):
            S = a[t][:, None, None] * S + (dm[t][:, None] * x[t])[..., None] * _heads(B[t], H)[:, None, :]
            y[t] = (S * _heads(C[t], H)[:, None, :]).sum(-1) + D[:, None] * x[t]
            kept.append(S)
        finals[i] = S
        if dy is None:
            continue
        T = f(dS[i]).clone() if dS is not None else torch.zeros_like(S)
        for t in reversed(range(s, e)):
            Bh, Ch = _heads(B[t], H), _heads(C[t], H)
            T = T + dy[t][..., None] * Ch[:, None, :]
            G = B.shape[1]
            g["dD"] += (dy[t] * x[t]).sum(-1)
            g["dC"][t] = (kept[t - s + 1] * dy[t][..., None]).sum(1).view(G, H // G, -1).sum(1)
            TB = (T * Bh[:, None, :]).sum(-1)
            g["dx"][t] = dm[t][:, None] * TB + D[:, None] * dy[t]
            g["dB"][t] = (dm[t][:, None] * (T * x[t][..., None]).sum(1)).view(G, H // G, -1).sum(1)
            dl = a[t] * (T * kept[t - s]).sum((1, 2))
            step = (Av * dl + (x[t] * TB).sum(-1)) * (torch.sigmoid(raw[t]) if sp else 1.0)
            g["ddt"][t] = step
            g["dA"] += dl * dm[t]
            g["ddt_bias"] += step
            T = a[t][:, None, None] * T
        g["dS0"][i] = T
    return y, finals, g


def gated(x, z, w, group, norm_first, eps, dy=None):
    x, z, w = (t.double().requires_grad_() for t in (x, z, w))
    gate = z / (1 + torch.exp(-z))
    u = x if norm_first else x * gate
    v = u.view(u.shape[0], u.shape[1] // group, group)
    y = (v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)).reshape(u.shape) * w
    y = y * gate if norm_first else y
    if dy is None:
        return y.detach()
    return (y.detach(), *torch.autograd.grad(y, (x, z, w), dy.double()))


def residual(x, r, w, scale, eps, dy=None, dr=None):
    """(y, stored sum[, dx, dr, dw]); the norm reads the sum as it is stored."""
    total = r.double() + scale * x.double()
    h, w = total.to(r.dtype).double().requires_grad_(), w.double().requires_grad_()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * w
    if dy is None:
        return y.detach(), total
    gh, gw = torch.autograd.grad(y, (h, w), dy.double())
    gh = gh + (dr.double() if dr is not None else 0)
    return y.detach(), total, scale * gh, gh, gw
