"""Plain float64 references of the block operators, on the CPU: definitions, token by token."""
from __future__ import annotations

import torch


def delta_fwd(q, k, v, g, beta, scale, S0=None):
    """One sequence.  q, k (L, Hk, K), v (L, H, V), g, beta (L, H), S0 (H, K, V), all float64.
    Returns o, the last state and every state (before each token, then the last)."""
    L, H, V = v.shape
    r = H // q.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    S = torch.zeros(H, q.shape[2], V, dtype=v.dtype) if S0 is None else S0.clone()
    o, states = torch.zeros_like(v), []
    for t in range(L):
        states.append(S)
        S = g[t].exp()[:, None, None] * S
        e = v[t] - (S * k[t][:, :, None]).sum(1)
        S = S + k[t][:, :, None] * (beta[t][:, None] * e)[:, None, :]
        o[t] = scale * (S * q[t][:, :, None]).sum(1)
    states.append(S)
    return o, S, states


def delta_bwd(q, k, v, g, beta, scale, do, S0=None, dlast=None):
    """Adjoints of delta_fwd, token by token: dq, dk, dv, dg, dbeta, dS0."""
    L, H, V = v.shape
    Hk, K = q.shape[1:]
    r = H // Hk
    _, S, states = delta_fwd(q, k, v, g, beta, scale, S0)
    qr, kr = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    dq, dk = torch.zeros_like(qr), torch.zeros_like(kr)
    dv, dg, db = torch.zeros_like(v), torch.zeros_like(g), torch.zeros_like(beta)
    dS = torch.zeros_like(S) if dlast is None else dlast.clone()
    for t in reversed(range(L)):
        a = g[t].exp()[:, None, None]
        Sa = a * states[t]
        dq[t] = scale * (states[t + 1] * do[t][:, None, :]).sum(2)
        dS = dS + scale * qr[t][:, :, None] * do[t][:, None, :]
        e = v[t] - (Sa * kr[t][:, :, None]).sum(1)
        w = (dS * kr[t][:, :, None]).sum(1)
        db[t] = (w * e).sum(1)
        dv[t] = beta[t][:, None] * w
        dk[t] = (dS * (beta[t][:, None] * e)[:, None, :]).sum(2) - (Sa * dv[t][:, None, :]).sum(2)
        dS = dS - kr[t][:, :, None] * dv[t][:, None, :]
        dg[t] = (dS * Sa).sum((1, 2))
        dS = a * dS
    fold = lambda x: x.reshape(L, Hk, r, K).sum(2)
    return dict(dq=fold(dq), dk=fold(dk), dv=dv, dg=dg, dbeta=db, dS0=dS)


def norm_fwd(x, w, b, eps):
    mean = x.mean(1)
    rstd = 1 / ((x - mean[:, None]).square().mean(1) + eps).sqrt()
    y = (x - mean[:, None]) * rstd[:, None]
    if w is not None:
        y = y * w
    return (y if b is None else y + b), mean, rstd


def norm_bwd(x, w, dy, mean, rstd):
    xh = (x - mean[:, None]) * rstd[:, None]
    u = dy if w is None else dy * w
    dx = rstd[:, None] * (u - u.mean(1, keepdim=True) - xh * (u * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
