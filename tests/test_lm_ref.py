"""The float64 references' gradients against automatic differentiation and against differences."""
import torch

import lm_ref

EPS = 1e-5


def rnd(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed + sum(s)), dtype=torch.float64)


def differences(f, x, h=1e-6):
    """Central differences of a scalar function."""
    d = torch.zeros_like(x)
    for i in range(x.numel()):
        e = torch.zeros_like(x).view(-1)
        e[i] = h
        d.view(-1)[i] = (f(x + e.view_as(x)) - f(x - e.view_as(x))) / (2 * h)
    return d


def test_block_norm_gradients():
    r, o, z, dy, dr = (rnd(3, 7, seed=i) for i in range(5))
    w, pw = rnd(7, seed=6), rnd(7, seed=7)

    def loss(r, w, o, pw, z):
        ro, y, *_ = lm_ref.block_norm_fwd(r, w, o, pw, z, 0.6, EPS)
        return (dy * y).sum() + (dr * ro).sum()

    ro, _, rstd, q = lm_ref.block_norm_fwd(r, w, o, pw, z, 0.6, EPS)
    d = lm_ref.block_norm_bwd(ro, dy, rstd, w, o, q, pw, z, 0.6, dr)
    args = [t.clone().requires_grad_() for t in (r, w, o, pw, z)]
    auto = torch.autograd.grad(loss(*args), args)
    for n, a in zip(("dr", "dweight", "do", "dpost_weight", "dz"), auto):
        assert torch.allclose(d[n], a, rtol=1e-10, atol=1e-12), n
    assert torch.allclose(d["do"], differences(lambda t: loss(r, w, t, pw, z), o), atol=1e-8)
    assert torch.allclose(d["dz"], differences(lambda t: loss(r, w, o, pw, t), z), atol=1e-8)
    d = lm_ref.block_norm_bwd(r, dy, lm_ref.rms(r, EPS)[1], w, dr_out=dr)
    f = lambda t: (dy * lm_ref.block_norm_fwd(t, w, eps=EPS)[1]).sum() + (dr * t).sum()
    assert torch.allclose(d["dr"], differences(f, r), atol=1e-8)


def test_xent_gradients():
    x, w = rnd(5, 6), rnd(9, 6)
    t = torch.tensor([3, -100, 8, 0, 9])
    dl, ds = rnd(5, seed=3), rnd(5, seed=4)

    def total(x, w):
        loss, lse, _ = lm_ref.xent_fwd(x, w, t, 0.7)
        return (dl * loss).sum() + (ds * lse).sum()

    _, lse, logits = lm_ref.xent_fwd(x, w, t, 0.7)
    g, _ = lm_ref.xent_g(logits, t, lse, dl, ds, 0.7)
    assert torch.allclose(g @ w, differences(lambda v: total(v, w), x), atol=1e-8)
    assert torch.allclose(g.t() @ x, differences(lambda v: total(x, v), w), atol=1e-8)
    assert bool((g[1] == 0).all()) and bool((g[4] == 0).all())


def test_embed_gradient():
    ids, dy = torch.tensor([2, 0, -1, 2, 5, 4]), rnd(6, 3)
    table = rnd(5, 3)
    f = lambda tb: (dy * lm_ref.embed_fwd(ids, tb, 1.5)).sum()
    d, _, _ = lm_ref.embed_bwd(ids, dy, 5, 1.5)
    assert torch.allclose(d, differences(f, table), atol=1e-8)
