"""Plain float64 references, on the CPU, of the embedding, the block norm and the linear cross entropy."""
from __future__ import annotations

import torch


def embed_fwd(ids, table, scale):
    y = torch.zeros(len(ids), table.shape[1], dtype=torch.float64)
    for t, i in enumerate(ids.tolist()):
        if 0 <= i < table.shape[0]:
            y[t] = scale * table[i]
    return y


def embed_bwd(ids, dy, V, scale):
    """dtable, and the sums of |scale dy| and the numbers of terms that a rounding bound takes."""
    ok = (ids >= 0) & (ids < V)
    d, size, n = (torch.zeros(V, dy.shape[1], dtype=torch.float64) for _ in range(3))
    d.index_add_(0, ids[ok], scale * dy[ok])
    size.index_add_(0, ids[ok], (scale * dy[ok]).abs())
    n.index_add_(0, ids[ok], torch.ones_like(dy[ok]))
    return d, size, n


def rms(x, eps):
    rstd = 1 / (x.square().mean(-1) + eps).sqrt()
    return x * rstd[..., None], rstd


def block_norm_fwd(r, w, o=None, pw=None, z=None, scale=1.0, eps=1e-5, held=None):
    """r_out (unrounded), y, rstd, post_rstd; held: the r_out that y is the norm of."""
    q = None
    if o is not None:
        a, q = rms(o, eps)
        a = a if pw is None else a * pw
        a = a if z is None else a * z / (1 + (-z).exp())
        r = r + scale * a
    y, rstd = rms(r if held is None else held, eps)
    return r, (y if w is None else y * w), rstd, q


def block_norm_bwd(r_out, dy, rstd, w=None, o=None, q=None, pw=None, z=None, scale=1.0, dr_out=None):
    rh = r_out * rstd[:, None]
    u = dy if w is None else dy * w
    G = rstd[:, None] * (u - rh * (u * rh).mean(1, keepdim=True))
    G = G if dr_out is None else G + dr_out
    d = {"dr": G, "dweight": (dy * rh).sum(0), "do": None, "dz": None, "dpost_weight": None}
    if o is not None:
        oh = o * q[:, None]
        a = oh if pw is None else oh * pw
        s = torch.ones_like(o) if z is None else torch.sigmoid(z)
        gate = s if z is None else z * s
        if z is not None:
            d["dz"] = scale * G * a * (s + z * s * (1 - s))
        c = scale * G * gate
        d["dpost_weight"] = (c * oh).sum(0)
        v = c if pw is None else c * pw
        d["do"] = q[:, None] * (v - oh * (v * oh).mean(1, keepdim=True))
    return d


def xent_fwd(x, w, targets, scale):
    """loss, lse, logits; rows without a target are zero in the first two."""
    V = w.shape[0]
    ok = (targets >= 0) & (targets < V)
    logits = scale * x @ w.t()
    lse = torch.logsumexp(logits, 1)
    at = logits.gather(1, targets.clamp(0, V - 1)[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    return torch.where(ok, lse - at, zero), torch.where(ok, lse, zero), logits


def xent_g(logits, targets, lse, dloss, dlse, scale):
    """Gradient of the unscaled products, and the part of it that is not the target's."""
    V = logits.shape[1]
    ok = (targets >= 0) & (targets < V)
    both = dloss if dlse is None else dloss + dlse
    p = scale * both[:, None] * (logits - lse[:, None]).exp()
    p = torch.where(ok[:, None], p, torch.zeros_like(p))
    one = torch.zeros_like(p)
    one[ok, targets[ok]] = scale * dloss[ok]
    return p - one, p
