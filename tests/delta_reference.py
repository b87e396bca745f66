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


def gradients(q, k, v, dt, b, A, bias, bounds, S0, dy, dS, *, scale=None, norm=True, beta=1.0, eps=1e-6, softplus=True):
    """(gradients, magnitudes) by the adjoint recurrence, dicts of dq, dk, dv, ddt, db, dA, ddt_bias, dS0.  The magnitudes of
    dq and dk are the sums of their terms' magnitudes that are made of decayed scores between two rows; of dl (entry
    "dl"): sums of |adjoint| |state|; of db: |F| |U|; of dS0: of what decays from the rows and from dS."""
    q, k, v, dt, b, A, S0, dy = (t.double() for t in (q, k, v, dt, b, A, S0, dy))
    R, H, P = v.shape
    G, N = k.shape[1:]
    scale = N ** -0.5 if scale is None else scale
    qh, kh = (unit(x, norm, eps).repeat_interleave(H // G, 1) for x in (q, k))
    raw = dt if bias is None else dt + bias.double()
    step = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    a, r = torch.exp(step * A), beta * torch.sigmoid(b)
    dyh = scale * dy
    zero = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    dqh, dkh, mq, mk = (zero(R, H, N) for _ in range(4))
    U, F = zero(R, H, P), zero(R, H, P)
    dl, ml, db, mb = (zero(R, H) for _ in range(4))
    dS0, mS = zero(*S0.shape), zero(*S0.shape)
    for i, (s, e) in enumerate(bounds):
        states = [S0[i]]
        for t in range(s, e):
            S = states[-1]
            U[t] = r[t][:, None] * (v[t] - a[t][:, None] * torch.matmul(S, kh[t][..., None])[..., 0])
            states.append(a[t][:, None, None] * S + U[t][..., None] * kh[t][:, None])
        T = zero(H, P, N) if dS is None else dS[i].double().clone()
        M = T.abs()
        for t in reversed(range(s, e)):
            S, S1 = states[t - s], states[t - s + 1]
            T = T + dyh[t][..., None] * qh[t][:, None]
            M = M + dyh[t].abs()[..., None] * qh[t].abs()[:, None]
            dqh[t] = torch.matmul(S1.transpose(1, 2), dyh[t][..., None])[..., 0]
            F[t] = torch.matmul(T, kh[t][..., None])[..., 0]  # what reaches r (v - a S k)
            de = r[t][:, None] * F[t]
            dkh[t] = (torch.matmul(T.transpose(1, 2), U[t][..., None])
                      - a[t][:, None, None] * torch.matmul(S.transpose(1, 2), de[..., None]))[..., 0]
            T = T - de[..., None] * kh[t][:, None]
            M = M + de.abs()[..., None] * kh[t].abs()[:, None]
            dl[t], ml[t] = a[t] * (T * S).sum((1, 2)), a[t] * (T.abs() * S.abs()).sum((1, 2))
            T, M = a[t][:, None, None] * T, a[t][:, None, None] * M
            db[t] = (F[t] * U[t]).sum(-1) * (1 - r[t] / beta)
            mb[t] = (F[t].abs() * U[t].abs()).sum(-1)
        dS0[i], mS[i] = T, M
        n = e - s
        if n:  # decays between rows i >= j, products of dY and U, of F and U
            L = torch.cumsum(step[s:e] * A, 0).T
            m = torch.exp((L[:, :, None] - L[:, None, :]).masked_fill(~torch.ones(n, n, dtype=torch.bool).tril(), -torch.inf))
            u, f, y = (t[s:e].transpose(0, 1) for t in (U, F, dyh))
            W = m * torch.matmul(y, u.transpose(1, 2)).abs()
            Y = m.tril(-1) * torch.matmul(f, u.transpose(1, 2)).abs() * r[s:e].T[:, :, None]
            ka, qa = kh[s:e].abs().transpose(0, 1), qh[s:e].abs().transpose(0, 1)
            mq[s:e] = torch.matmul(W, ka).transpose(0, 1)
            mk[s:e] = (torch.matmul(W.transpose(1, 2), qa) + torch.matmul(Y, ka) + torch.matmul(Y.transpose(1, 2), ka)).transpose(0, 1)

    def through(x, g, m):
        g, m = (t.view(R, G, H // G, N).sum(2) for t in (g, m))
        if not norm:
            return g, m
        inv = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) + eps)
        y = x * inv
        return inv * (g - y * (y * g).sum(-1, keepdim=True)), inv * (m + y.abs() * (y.abs() * m).sum(-1, keepdim=True))

    (dq, mq), (dk, mk) = through(q, dqh, mq), through(k, dkh, mk)
    slope = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
    ddt = A * dl * slope
    rows = [t for s, e in bounds for t in range(s, e)]
    g = dict(dq=dq, dk=dk, dv=r[..., None] * F, ddt=ddt, db=db, dA=(dl * step)[rows].sum(0), ddt_bias=ddt[rows].sum(0), dS0=dS0)
    return g, dict(dq=mq, dk=mk, dl=ml, db=mb, dS0=mS, slope=A.abs() * slope, step=step.abs())
