"""Measured cases of the gated delta rule, layer norm and gradient-clipping operators.

Each case names one operator and its sizes.  ``run`` computes it either with the package's HIP
entry points (``own`` true) or in a plain form of elementary torch operations in float32
(``own`` false); ``exact`` computes it from its definition in float64, token by token for the
recurrence.

The gated delta rule, per sequence and value head, with a state S of K x V and a log decay
g_t <= 0:

    e_t = v_t - exp(g_t) S_{t-1}^T k_t,   S_t = exp(g_t) S_{t-1} + beta_t k_t e_t^T,
    o_t = scale S_t^T q_t

Query / key head h // (H / Hk) serves value head h.  Packed cases hold several sequences of
different lengths (some empty) in one array, bounded by seq_offsets.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEVICE = "cuda"
CHUNK = 64        # tokens per block of the plain form's recurrence
EPS_NORM = 1e-5   # layer norm's epsilon
EPS_CLIP = 1e-6   # added to the norm in the clipping coefficient
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one short prompt of a small model: a call whose launches are most of its time
        dict(name="delta_fwd_tiny_f32", op="delta_fwd", io="f32", Bt=1, L=64, Hk=4, H=4, K=32, V=32,
             packed=0),
        # prefill of four prompts at the 4096-channel layer shape, two value heads per key head
        dict(name="delta_fwd_prefill_bf16", op="delta_fwd", io="bf16", Bt=4, L=4096, Hk=16, H=32,
             K=128, V=128, packed=0),
        # one very long document at the 2048-channel layer shape: few heads, many chunks
        dict(name="delta_fwd_long_bf16", op="delta_fwd", io="bf16", Bt=1, L=65536, Hk=16, H=16,
             K=128, V=128, packed=0),
        # a packed batch of ragged prompts (one empty, one of a single token), odd head sizes
        dict(name="delta_fwd_packed_f32", op="delta_fwd", io="f32", Bt=9, L=8191, Hk=3, H=6, K=96,
             V=80, packed=1),
        # a training backward at the fp32 2048-channel layer shape
        dict(name="delta_bwd_f32", op="delta_bwd", io="f32", Bt=4, L=2048, Hk=16, H=16, K=128,
             V=128, packed=0),
        # a training backward over packed documents, two value heads per key head
        dict(name="delta_bwd_packed_bf16", op="delta_bwd", io="bf16", Bt=12, L=16384, Hk=8, H=16,
             K=128, V=128, packed=1),
        # one token for one user: latency
        dict(name="delta_step_one_bf16", op="delta_step", io="bf16", Bt=1, Hk=16, H=16, K=128,
             V=128),
        # one token for a serving batch of 256 at the 4096-channel layer shape
        dict(name="delta_step_batch_bf16", op="delta_step", io="bf16", Bt=256, Hk=16, H=32, K=128,
             V=128),
        # the block's norm over four 4096-token sequences of 4096 channels, forward and backward
        dict(name="layer_norm_fwd_bf16", op="norm_fwd", io="bf16", rows=16384, D=4096),
        dict(name="layer_norm_bwd_bf16", op="norm_bwd", io="bf16", rows=16384, D=4096),
        # gradients of a small model: over a hundred little tensors, launches count
        dict(name="clip_small_f32", op="clip", io="f32", layers=16, D=129, clipped=1),
        # gradients of a 24-layer stack of 2048 channels
        dict(name="clip_stack_bf16", op="clip", io="bf16", layers=24, D=2048, clipped=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _head(rng, most):
    return rng.choice([16, 32, 64, 64, 96, 128, 128, 192, 256, rng.randrange(1, most + 1)])


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_bwd", "delta_bwd", "delta_step", "norm_fwd",
                     "norm_bwd", "clip"])
    io = rng.choice(["f32", "bf16"])
    if op in ("norm_fwd", "norm_bwd"):
        D = _log(rng, 16, 16384)
        return dict(op=op, io=io, rows=_log(rng, 1, max(2, (1 << 26) // D)), D=D)
    if op == "clip":
        return dict(op=op, io=io, layers=_log(rng, 1, 32), D=_log(rng, 16, 1536),
                    clipped=rng.randrange(2))
    Hk = _log(rng, 1, 16)
    H = Hk * rng.choice([1, 1, 2, 4])
    K, V = _head(rng, 256), _head(rng, 256)
    if op == "delta_step":
        most = max(2, (1 << 27) // (H * K * V))
        return dict(op=op, io=io, Bt=_log(rng, 1, most), Hk=Hk, H=H, K=K, V=V)
    budget = (1 << 32) if op == "delta_fwd" else (1 << 31)
    tokens = max(2, min(32768, budget // (H * max(K, 64) * max(V, 64))))
    packed = int(rng.random() < 0.4)
    if packed:
        return dict(op=op, io=io, Bt=rng.randrange(1, 17), L=_log(rng, 1, tokens), Hk=Hk, H=H, K=K,
                    V=V, packed=1)
    L = _log(rng, 1, tokens)
    return dict(op=op, io=io, Bt=_log(rng, 1, max(1, min(16, tokens // L))), L=L, Hk=Hk, H=H, K=K,
                V=V, packed=0)


def _lengths(case):
    """Lengths of a packed case's sequences: they sum to L; an empty and a one-token sequence are
    among them when there are enough sequences."""
    r = random.Random(case["Bt"] * 1000003 + case["L"])
    n, total = case["Bt"], case["L"]
    fixed = ([0] if n >= 4 else []) + ([1] if n >= 3 and total > 1 else [])
    rest = n - len(fixed)
    cuts = sorted(r.randrange(total - sum(fixed) + 1) for _ in range(rest - 1))
    ends = cuts + [total - sum(fixed)]
    got = [b - a for a, b in zip([0] + cuts, ends)] + fixed
    r.shuffle(got)
    return got


def _clip_shapes(case):
    """Parameter shapes of `layers` blocks of width D: two projections, a short filter and five
    per-channel or per-head vectors each."""
    D = case["D"]
    block = [(2 * D, D), (D, D), (D, 4), (D,), (D,), (D,), (max(1, D // 128),), (16, D)]
    return block * case["layers"]


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    dt = DTYPES[case["io"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=DEVICE)

    op = case["op"]
    s = {"case": case, "op": op}
    if op in ("norm_fwd", "norm_bwd"):
        rows, D = case["rows"], case["D"]
        # activations of a residual stream: a per-channel offset and scale
        x = normal(rows, D) * (0.5 + uniform(D)) + 0.3 * normal(D)
        s.update(x=x.to(dt), weight=1 + 0.1 * normal(D), bias=0.1 * normal(D))
        if op == "norm_bwd":
            s["dy"] = normal(rows, D).to(dt)
            xf = s["x"].float()
            mean = xf.mean(1)
            var = (xf - mean[:, None]).square().mean(1)
            s.update(mean=mean, rstd=torch.rsqrt(var + EPS_NORM))
        return s
    if op == "clip":
        grads = [(0.01 * normal(*shape)).to(dt) for shape in _clip_shapes(case)]
        numel = sum(t.numel() for t in grads)
        # the clipped gradients go into one flat buffer, each at a multiple of 64 elements
        starts = [0]
        for t in grads:
            starts.append(starts[-1] + -(-t.numel() // 64) * 64)
        flat = torch.zeros(starts[-1], dtype=dt, device=DEVICE)
        out = [flat[a : a + t.numel()].view(t.shape) for a, t in zip(starts, grads)]
        # half of the expected norm when the gradients are to be clipped, twice it otherwise
        s.update(grads=grads, out=out, flat=flat, starts=starts,
                 max_norm=0.01 * math.sqrt(numel) * (0.5 if case["clipped"] else 2.0))
        return s
    Bt, Hk, H, K, V = (case[n] for n in ("Bt", "Hk", "H", "K", "V"))
    if op == "delta_step":
        lead, n = (Bt,), Bt
    elif case["packed"]:
        lead, n = (case["L"],), case["Bt"]
    else:
        lead, n = (Bt, case["L"]), Bt

    def unit(*shape):  # rows of length one, as queries and keys are normalised
        x = normal(*shape)
        return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)).to(dt)

    # decay of a selective layer: a rate per head times a step between 1e-3 and 1e-1
    rate = 1 + 15 * uniform(H)
    step = torch.exp(math.log(1e-3) + math.log(100.0) * uniform(*lead, H))
    s.update(q=unit(*lead, Hk, K), k=unit(*lead, Hk, K), v=normal(*lead, H, V).to(dt),
             g=-rate * step, beta=torch.sigmoid(normal(*lead, H)), scale=K ** -0.5)
    s["S"] = 0.3 * normal(n, H, K, V)
    if op == "delta_step":
        return s
    s["seq_offsets"] = None
    if case["packed"]:
        ends = [0]
        for l in _lengths(case):
            ends.append(ends[-1] + l)
        s["seq_offsets"] = torch.tensor(ends, dtype=torch.int32, device=DEVICE)
        s["longest"] = max(_lengths(case))
    if op == "delta_bwd":
        s["do"] = normal(*lead, H, V).to(dt)
        s["dlast_S"] = normal(n, H, K, V)
    return s


# ---- the plain forms -----------------------------------------------------------------------

def _unit_lower_inverse(M):
    """Inverse of I + M for strictly lower M (..., C, C), C a power of two: the inverses of the
    diagonal blocks are joined in pairs, -T2 M21 T1 being the block below."""
    C = M.shape[-1]
    T = torch.eye(C, dtype=M.dtype, device=M.device).expand(M.shape)
    n = 1
    at = torch.arange(C, device=M.device)
    while n < C:
        below = ((at[:, None] // n) % 2 == 1) & (at[None, :] // n == at[:, None] // n - 1)
        T = T - T @ (M * below) @ T
        n *= 2
    return T


def _plain_delta(q, k, v, g, beta, S, scale):
    """q, k, v (B, L, H, .), g, beta (B, L, H), S (B, H, K, V), all float32.  Blocks of CHUNK
    tokens: within a block the recurrence is a unit lower triangular system, solved for every
    block at once; the state passes from block to block."""
    B, L, H, V = v.shape
    n = -(-L // CHUNK)

    def blocks(x):
        x = torch.nn.functional.pad(x.transpose(1, 2).flatten(3), (0, 0, 0, n * CHUNK - L))
        return x.reshape(B, H, n, CHUNK, -1)

    q, k, v = blocks(q), blocks(k), blocks(v)
    G = blocks(g[..., None])[..., 0].cumsum(-1)
    beta = blocks(beta[..., None])
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    D = torch.where(lower, (G[..., :, None] - G[..., None, :]).masked_fill(~lower, 0.0).exp(), 0.0)
    kt = k.transpose(-1, -2)
    T = _unit_lower_inverse((k @ kt * D * beta).tril(-1))
    P = q @ kt * D * scale
    U, W = T @ (beta * v), T @ (beta * G.exp()[..., None] * k)
    qg = q * (G.exp()[..., None] * scale)
    kw = (k * (G[..., -1:] - G).exp()[..., None]).transpose(-1, -2)
    last = G[..., -1].exp()[..., None, None]
    out = []
    for c in range(n):
        u = U[:, :, c] - W[:, :, c] @ S
        out.append(qg[:, :, c] @ S + P[:, :, c] @ u)
        S = last[:, :, c] * S + kw[:, :, c] @ u
    o = torch.stack(out, 2).reshape(B, H, n * CHUNK, V)[:, :, :L]
    return o.transpose(1, 2), S


def _plain_delta_any(q, k, v, g, beta, S, scale, offsets, longest):
    H = v.shape[-2]

    def heads(x):  # each key head serves H / Hk value heads
        return x.repeat_interleave(H // x.shape[-2], dim=-2)

    q, k = heads(q), heads(k)
    if offsets is None:
        return _plain_delta(q, k, v, g, beta, S, scale)
    # packed: sequences side by side, padded with tokens that change nothing
    n, longest = offsets.numel() - 1, max(longest, 1)
    token = torch.arange(v.shape[0], device=v.device)
    seq = torch.searchsorted(offsets[1:].long(), token, right=True)
    at = seq * longest + token - offsets.long()[seq]

    def side_by_side(x):
        y = x.new_zeros((n * longest,) + x.shape[1:]).index_copy(0, at, x)
        return y.reshape((n, longest) + x.shape[1:])

    o, S = _plain_delta(*(side_by_side(x) for x in (q, k, v, g, beta)), S, scale)
    return o.reshape((n * longest,) + o.shape[2:]).index_select(0, at), S


def _plain_norm(x, weight, bias):
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt(c.square().mean(1) + EPS_NORM)
    return c * rstd[:, None] * weight + bias, mean, rstd


def _run_plain(s):
    op = s["op"]
    if op == "norm_fwd":
        y, mean, rstd = _plain_norm(s["x"].float(), s["weight"], s["bias"])
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dy = s["dy"].float()
        xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        w = dy * s["weight"]
        dx = s["rstd"][:, None] * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}
    if op == "clip":
        wide = [t.float() for t in s["grads"]]
        norm = torch.stack([t.square().sum() for t in wide]).sum().sqrt()
        coef = (s["max_norm"] / (norm + EPS_CLIP)).clamp_max(1.0)
        for o, t in zip(s["out"], wide):
            o.copy_(t * coef)
        return {"norm": norm, "clipped": s["flat"]}
    if op == "delta_step":
        H = s["v"].shape[1]
        q, k = (s[n].float().repeat_interleave(H // s[n].shape[1], 1)[..., None] for n in "qk")
        S = s["S"] * s["g"].exp()[..., None, None]
        e = s["beta"][..., None] * (s["v"].float() - (S * k).sum(-2))
        S = S + k * e[..., None, :]
        s["S"].copy_(S)
        return {"o": (s["scale"] * (S * q).sum(-2)).to(s["v"].dtype), "S": s["S"]}
    args = [s[n].float() for n in ("q", "k", "v", "g", "beta", "S")]
    where = (s["scale"], s["seq_offsets"], s.get("longest"))
    if op == "delta_fwd":
        o, S = _plain_delta_any(*args, *where)
        return {"o": o.to(s["v"].dtype), "last_S": S}
    args = [a.detach().requires_grad_() for a in args]
    o, S = _plain_delta_any(*args, *where)
    grads = torch.autograd.grad([o, S], args, [s["do"].float(), s["dlast_S"]])
    io = s["v"].dtype
    names = ("dq", "dk", "dv", "dg", "dbeta", "dS0")
    return {n: d.to(io) if n in ("dq", "dk", "dv") else d for n, d in zip(names, grads)}


def _run_own(s):
    import selective_state_space_msm_amd as msm
    op = s["op"]
    if op == "norm_fwd":
        y, mean, rstd = msm.msm_layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=EPS_NORM,
                                               return_stats=True)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        return msm.msm_layer_norm_bwd(s["x"], s["dy"], s["mean"], s["rstd"], s["weight"],
                                      bias_grad=True)
    if op == "clip":
        norm = msm.msm_grad_clip(s["grads"], s["max_norm"], eps=EPS_CLIP, out=s["out"])
        return {"norm": norm, "clipped": s["flat"]}
    if op == "delta_step":
        o = msm.msm_delta_rule_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S"],
                                    s["scale"])
        return {"o": o, "S": s["S"]}
    if op == "delta_fwd":
        o, S = msm.msm_delta_rule_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"],
                                      S0=s["S"], seq_offsets=s["seq_offsets"],
                                      return_last_state=True)
        return {"o": o, "last_S": S}
    return msm.msm_delta_rule_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], s["scale"],
                                  S0=s["S"], dlast_S=s["dlast_S"], seq_offsets=s["seq_offsets"],
                                  state_grads=True)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- definitions in 64 bits ------------------------------------------------------------------

def _exact_steps(q, k, v, g, beta, S, scale, keep=None):
    """The recurrence token by token; q, k (L, B, H, K), v (L, B, H, V), g, beta (L, B, H).
    `keep`: a list that receives every state before its token."""
    a = g.exp()
    out = torch.empty_like(v)
    for t in range(v.shape[0]):
        if keep is not None:
            keep.append(S)
        S = a[t][..., None, None] * S
        e = v[t] - torch.matmul(k[t][..., None, :], S)[..., 0, :]
        S = S + k[t][..., :, None] * (beta[t][..., None] * e)[..., None, :]
        out[t] = scale * torch.matmul(q[t][..., None, :], S)[..., 0, :]
    return out, S


def _exact_steps_back(q, k, v, g, beta, S, scale, do, dS):
    """Adjoints of _exact_steps, walking back through the tokens; states are kept for one block
    of tokens at a time."""
    L = v.shape[0]
    starts, s = [], S
    for c in range(0, L, CHUNK):
        starts.append(s)
        e = slice(c, c + CHUNK)
        _, s = _exact_steps(q[e], k[e], v[e], g[e], beta[e], s, scale)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(g), torch.zeros_like(beta)
    for c in reversed(range(0, L, CHUNK)):
        e, keep = slice(c, c + CHUNK), []
        _, s_end = _exact_steps(q[e], k[e], v[e], g[e], beta[e], starts[c // CHUNK], scale, keep)
        keep.append(s_end)
        for t in reversed(range(c, min(c + CHUNK, L))):
            before, after = keep[t - c], keep[t - c + 1]
            kt, at, bt = k[t][..., :, None], g[t].exp()[..., None, None], beta[t][..., None]
            dq[t] = scale * torch.matmul(after, do[t][..., :, None])[..., 0]
            dS = dS + scale * q[t][..., :, None] * do[t][..., None, :]
            err = v[t] - torch.matmul(k[t][..., None, :], at * before)[..., 0, :]
            w = torch.matmul(k[t][..., None, :], dS)[..., 0, :]        # adjoint of beta * err
            db[t] = (w * err).sum(-1)
            dv[t] = bt * w
            dk[t] = (torch.matmul(dS, (bt * err)[..., :, None])
                     - torch.matmul(at * before, dv[t][..., :, None]))[..., 0]
            dS = dS - kt * dv[t][..., None, :]                          # adjoint of the decayed state
            dg[t] = (dS * (at * before)).sum((-1, -2))
            dS = at * dS
    return dq, dk, dv, dg, db, dS


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    w = {n: t.double() for n, t in s.items() if torch.is_tensor(t) and t.is_floating_point()}
    if op == "norm_fwd":
        x = w["x"]
        mean, var = x.mean(1), x.var(1, unbiased=False)
        rstd = (var + EPS_NORM) ** -0.5
        y = (x - mean[:, None]) * rstd[:, None]
        return {"y": y * w["weight"] + w["bias"], "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        D = w["x"].shape[1]
        xh = (w["x"] - w["mean"][:, None]) * w["rstd"][:, None]
        wdy = w["dy"] * w["weight"]
        a, b = wdy.sum(1, keepdim=True) / D, (wdy * xh).sum(1, keepdim=True) / D
        return {"dx": (wdy - a - b * xh) * w["rstd"][:, None], "dweight": (w["dy"] * xh).sum(0),
                "dbias": w["dy"].sum(0)}
    if op == "clip":
        flat = torch.zeros(s["starts"][-1], dtype=torch.float64, device=DEVICE)
        for a, t in zip(s["starts"], s["grads"]):
            flat[a : a + t.numel()] = t.double().reshape(-1)
        norm = flat.dot(flat) ** 0.5
        return {"norm": norm, "clipped": flat * min(1.0, s["max_norm"] / (float(norm) + EPS_CLIP))}
    H, Hk = s["v"].shape[-2], s["q"].shape[-2]
    r = H // Hk
    q, k = (w[n].repeat_interleave(r, -2) for n in "qk")
    if op == "delta_step":
        o, S = _exact_steps(q[None], k[None], w["v"][None], w["g"][None], w["beta"][None], w["S"],
                            s["scale"])
        return {"o": o[0], "S": S}
    if case["packed"]:
        # sequences side by side: a token past a sequence's end has g = beta = k = q = 0
        ends = s["seq_offsets"].tolist()
        longest = max(1, s["longest"])

        def spread(x):
            y = x.new_zeros((longest, len(ends) - 1) + x.shape[1:])
            for b, (lo, hi) in enumerate(zip(ends, ends[1:])):
                y[: hi - lo, b] = x[lo:hi]
            return y

        def gather(y):
            return torch.cat([y[: hi - lo, b] for b, (lo, hi) in enumerate(zip(ends, ends[1:]))])
    else:
        def spread(x):
            return x.transpose(0, 1)

        def gather(y):
            return y.transpose(0, 1)
    ins = [spread(x).contiguous() for x in (q, k, w["v"], w["g"], w["beta"])]
    if op == "delta_fwd":
        o, S = _exact_steps(*ins, w["S"], s["scale"])
        return {"o": gather(o), "last_S": S}
    d = _exact_steps_back(*ins, w["S"], s["scale"], spread(w["do"]).contiguous(), w["dlast_S"])
    dq, dk = (gather(x) for x in d[:2])
    dq, dk = (x.reshape(x.shape[:-2] + (Hk, r, x.shape[-1])).sum(-2) for x in (dq, dk))
    return dict(dq=dq, dk=dk, dv=gather(d[2]), dg=gather(d[3]), dbeta=gather(d[4]), dS0=d[5])


def work(case):
    """Each input read once and each output written once; operations of the definitions (the
    recurrence's 6 K V per token and head: the prediction, the write and the readout)."""
    es = 2 if case["io"] == "bf16" else 4
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        n, D = case["rows"] * case["D"], case["D"]
        if op == "norm_fwd":
            return {"bytes": 2 * n * es + 8 * D + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * es + 12 * D + 8 * case["rows"], "flops": 14 * n}
    if op == "clip":
        n = sum(math.prod(shape) for shape in _clip_shapes(case))
        return {"bytes": 2 * n * es + 4, "flops": 3 * n}
    Bt, Hk, H, K, V = (case[n] for n in ("Bt", "Hk", "H", "K", "V"))
    state = 4 * Bt * H * K * V
    if op == "delta_step":
        token = (2 * Hk * K + 2 * H * V) * es + 8 * H
        return {"bytes": Bt * token + 2 * state, "flops": 7 * Bt * H * K * V}
    tokens = case["L"] if case["packed"] else Bt * case["L"]
    if op == "delta_fwd":
        return {"bytes": tokens * ((2 * Hk * K + 2 * H * V) * es + 8 * H) + 2 * state,
                "flops": 6 * tokens * H * K * V}
    # backward: the states again (4 K V), the adjoint state (6 K V), dq and dk (6 K V)
    return {"bytes": tokens * ((4 * Hk * K + 3 * H * V) * es + 16 * H) + 3 * state,
            "flops": 16 * tokens * H * K * V}
