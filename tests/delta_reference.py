"""The gated delta rule in float64 from its definition, one row at a time (CPU).  Gradients by differentiating it."""
import torch


def _heads(t, H):
    return t.repeat_interleave(H // t.shape[0], 0)


def unit(x, norm, eps):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + eps) if norm else x


def rule(q, k, v, dt, b, A, bias, bounds, S0, *, scale=None, norm=True, beta=1.0, eps=1e-6, softplus=True):
    """(y, final states, magnitudes): bounds [(first row, end row)] of the sequences, S0 [nseq, H, P, N].  The magnitudes
    are those of y's terms and of the final states' terms: sums of |u| |k| |q|, decayed, with u as it comes out."""
    q, k, v, dt, b, A, S0 = (t.double() for t in (q, k, v, dt, b, A, S0))
    R, H, P = v.shape
    N = k.shape[2]
    scale = N ** -0.5 if scale is None else scale
    q, k = unit(q, norm, eps), unit(k, norm, eps)
    raw = dt if bias is None else dt + bias.double()
    step = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    a, r = torch.exp(step * A), beta * torch.sigmoid(b)
    ys, mags, finals, state_mags = {}, torch.zeros(R, H, P, dtype=torch.float64), [], []
    for i, (s, e) in enumerate(bounds):
        S, M = S0[i], S0[i].detach().abs()
        for t in range(s, e):
            kt, qt, at = _heads(k[t], H), _heads(q[t], H), a[t][:, None]
            u = r[t][:, None] * (v[t] - at * (S * kt[:, None]).sum(-1))
            S = at[..., None] * S + u[..., None] * kt[:, None]
            ys[t] = scale * (S * qt[:, None]).sum(-1)
            with torch.no_grad():
                M = at[..., None] * M + u.abs()[..., None] * kt.abs()[:, None]
                mags[t] = abs(scale) * (M * qt.abs()[:, None]).sum(-1)
        finals.append(S)
        state_mags.append(M)
    y = torch.stack([ys[t] if t in ys else torch.zeros(H, P, dtype=torch.float64) for t in range(R)])
    finals, state_mags = (torch.stack(f) if f else S0 for f in (finals, state_mags))
    return y, finals, (mags, state_mags)
