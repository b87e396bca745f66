"""The reference of the delta rule's gradients (CPU): the adjoint recurrence against automatic differentiation of the
definition in float64, and against central differences of it."""
import pytest

torch = pytest.importorskip("torch")

import delta_reference as ref  # noqa: E402

CASES = [dict(), dict(norm=False, beta=1.5), dict(softplus=False), dict(scale=1.0, eps=0.1)]


def problem(seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    R, H, P, G, N = 14, 4, 3, 2, 5
    t = dict(q=rnd(R, G, N), k=rnd(R, G, N) * 0.5, v=rnd(R, H, P), dt=rnd(R, H).abs() * 0.3, b=rnd(R, H),
             A=-rnd(H).abs(), bias=rnd(H).abs() * 0.1)
    return t, [(0, 9), (9, 9), (9, 14)], rnd(3, H, P, N), rnd(R, H, P), rnd(3, H, P, N)


@pytest.mark.parametrize("kw", CASES, ids=str)
def test_gradients(kw):
    t, bounds, S0, dy, dS = problem()
    leaves = [x.clone().requires_grad_() for x in (*t.values(), S0)]

    def loss(args):
        y, final, _ = ref.rule(*args[:7], bounds, args[7], **kw)
        return (y * dy).sum() + (final * dS).sum()

    auto = torch.autograd.grad(loss(leaves), leaves)
    g, _ = ref.gradients(*t.values(), bounds, S0, dy, dS, **kw)
    names = ("dq", "dk", "dv", "ddt", "db", "dA", "ddt_bias", "dS0")
    for name, want in zip(names, auto):
        assert torch.allclose(g[name], want, rtol=1e-10, atol=1e-12), name
    gen = torch.Generator().manual_seed(7)
    for n, name in enumerate(names):
        e = torch.randn(leaves[n].shape, generator=gen, dtype=torch.float64)
        args = [x.detach() for x in leaves]
        up, down = (loss([*args[:n], args[n] + s * 1e-6 * e, *args[n + 1:]]) for s in (1, -1))
        assert abs(float((g[name] * e).sum() - (up - down) / 2e-6)) < 1e-6, name
