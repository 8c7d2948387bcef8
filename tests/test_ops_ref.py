"""The float64 references of the block operators against central differences (CPU)."""
import torch

import ops_ref


def _differences(f, args, grads, eps=1e-6, picks=12, seed=0):
    """Directional derivatives of f along random directions of each argument."""
    gen = torch.Generator().manual_seed(seed)
    for i, (a, d) in enumerate(zip(args, grads)):
        for _ in range(picks // len(args) + 1):
            u = torch.randn(a.shape, generator=gen, dtype=a.dtype)
            up = f(*args[:i], a + eps * u, *args[i + 1:])
            dn = f(*args[:i], a - eps * u, *args[i + 1:])
            want = float((up - dn) / (2 * eps))
            got = float((d * u).sum())
            # truncation eps^2 and rounding 1e-16 / eps of terms of size ~ |f|
            assert abs(got - want) <= 1e-6 * max(1.0, abs(want)), (i, got, want)


def test_delta_gradients():
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    L, Hk, H, K, V = 9, 2, 4, 5, 6
    q, k, v = rnd(L, Hk, K), rnd(L, Hk, K) / K ** 0.5, rnd(L, H, V)
    g, beta = -rnd(L, H).abs(), torch.sigmoid(rnd(L, H))
    S0, do, dl = rnd(H, K, V), rnd(L, H, V), rnd(H, K, V)

    def loss(q, k, v, g, beta, S0):
        o, S, _ = ops_ref.delta_fwd(q, k, v, g, beta, 0.7, S0)
        return (o * do).sum() + (S * dl).sum()

    d = ops_ref.delta_bwd(q, k, v, g, beta, 0.7, do, S0, dl)
    _differences(loss, [q, k, v, g, beta, S0], [d[n] for n in ("dq", "dk", "dv", "dg", "dbeta", "dS0")])


def test_norm_gradients():
    gen = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    x, w, b, dy = rnd(5, 24), 1 + 0.3 * rnd(24), rnd(24), rnd(5, 24)

    def loss(x, w, b):
        return (ops_ref.norm_fwd(x, w, b, 1e-3)[0] * dy).sum()

    _, mean, rstd = ops_ref.norm_fwd(x, w, b, 1e-3)
    _differences(loss, [x, w, b], ops_ref.norm_bwd(x, w, dy, mean, rstd))
