"""Measured cases of the operators at a language model's ends and between its blocks: the token
embedding with its gradient, the norms around a block fused with its gate and residual scale, and
the cross entropy over a vocabulary that never keeps the logits.

Each case names one operator and its sizes.  ``run`` computes it either with the package's HIP
entry points (``own`` true) or in a plain form of elementary torch operations in float32 (``own``
false); ``exact`` computes it from its definition in float64.

Embedding, for a token id in [0, V) (any other id: a row of zeros, and nothing in the gradient):
    y_t = scale table[id_t],            dtable[v] = scale sum over {t: id_t = v} of dy_t
Block norm, with RMS(x) = x / sqrt(mean(x^2) + eps) over the last dimension:
    r'_t = r_t + scale post_weight RMS(o_t) silu(z_t),      y_t = weight RMS(r'_t)
    (no z: no gate; no o: r' = r).  r' is held in the I/O type and y is the norm of what is held.
Linear cross entropy, for a target in [0, V) (any other target: the row is left out, its loss, lse
and gradient are zero):
    l_tv = scale x_t . W_v,   lse_t = log sum_v exp(l_tv),   loss_t = lse_t - l_t,target
    backward of sum(dloss loss) + sum(dlse lse), from the forward's lse:
    g_tv = scale ((dloss_t + dlse_t) exp(l_tv - lse_t) - dloss_t [v = target_t]),
    dx = g W,   dW = g^T x
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the next tokens of a serving batch of 256 sequences, 4096-channel model: latency
        dict(name="embed_fwd_tokens_bf16", op="embed_fwd", table="bf16", io="bf16", T=256, V=65536, D=4096),
        # a training batch of four 4096-token sequences out of an fp32 master table
        dict(name="embed_fwd_batch_f32_bf16", op="embed_fwd", table="f32", io="bf16", T=16384, V=50000, D=2048),
        # the same batch's gradient: frequent tokens, rare ones, padding
        dict(name="embed_bwd_batch_bf16", op="embed_bwd", table="bf16", io="bf16", T=16384, V=65536, D=2048),
        # gradient of a small model's embedding in odd sizes
        dict(name="embed_bwd_small_f32", op="embed_bwd", table="f32", io="f32", T=2047, V=1003, D=129),
        # one token between two blocks of a 4096-channel model: latency
        dict(name="block_norm_fwd_token_bf16", op="block_norm_fwd", io="bf16", rows=1, D=4096, block=1, gate=1),
        # four 4096-token sequences between two gated blocks, forward and backward
        dict(name="block_norm_fwd_bf16", op="block_norm_fwd", io="bf16", rows=16384, D=4096, block=1, gate=1),
        dict(name="block_norm_bwd_bf16", op="block_norm_bwd", io="bf16", rows=16384, D=4096, block=1, gate=1),
        # a small fp32 model's backward, no gate, odd sizes
        dict(name="block_norm_bwd_odd_f32", op="block_norm_bwd", io="f32", rows=4095, D=1001, block=1, gate=0),
        # log-probabilities of one token each of 16 served sequences: the weights are most of the bytes
        dict(name="xent_fwd_serve_bf16", op="xent_fwd", io="bf16", T=16, V=65536, D=4096, ignored=0.0),
        # the loss of 8192 training tokens over a large vocabulary, some of them padding
        dict(name="xent_fwd_batch_bf16", op="xent_fwd", io="bf16", T=8192, V=65536, D=2048, ignored=0.05),
        # its backward, with the gradient of a penalty on lse beside the loss's
        dict(name="xent_bwd_batch_bf16", op="xent_bwd", io="bf16", T=8192, V=65536, D=2048, ignored=0.05, penalty=1),
        # the backward of a small fp32 model, odd sizes, half of the tokens without a target
        dict(name="xent_bwd_odd_f32", op="xent_bwd", io="f32", T=1999, V=10007, D=513, ignored=0.5, penalty=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _some(rng, lo, hi):
    """A size of the range: half the time any, half the time a multiple of 64 where one fits."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.5 or n < 64 else n // 64 * 64


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "embed_bwd", "block_norm_fwd", "block_norm_bwd",
                     "xent_fwd", "xent_fwd", "xent_bwd", "xent_bwd"])
    io = rng.choice(["f32", "bf16"])
    D = _some(rng, 16, 8192)
    if op.startswith("embed"):
        V = _some(rng, 64, max(65, min(1 << 18, (1 << 27) // D)))
        return dict(op=op, table=rng.choice(["f32", io]), io=io, T=_some(rng, 1, max(2, min(1 << 17, (1 << 25) // D))),
                    V=V, D=D)
    if op.startswith("block_norm"):
        block = int(rng.random() < 0.8)
        return dict(op=op, io=io, rows=_some(rng, 1, max(2, (1 << 25) // D)), D=D, block=block,
                    gate=block * rng.randrange(2))
    V = _some(rng, 64, min(1 << 17, (1 << 28) // D))
    products = 1 << (39 if io == "bf16" else 36)
    T = _some(rng, 1, max(2, min(16384, products // (V * D), (1 << 29) // V)))
    return dict(op=op, io=io, T=T, V=V, D=D, ignored=rng.choice([0.0, 0.0, 0.1, 0.5]), penalty=rng.randrange(2))


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    dt = DTYPES[case["io"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=DEVICE)

    op, D = case["op"], case["D"]
    s = {"case": case, "op": op}
    if op.startswith("embed"):
        T, V = case["T"], case["V"]
        # a token's frequency falls as one over its rank; one position in 32 is padding
        ids = (V ** uniform(T).double()).long().sub(1).clamp(0, V - 1)
        s.update(ids=torch.where(uniform(T) < 1 / 32, -1, ids), V=V, scale=math.sqrt(D), table_dtype=DTYPES[case["table"]])
        if op == "embed_fwd":
            s.update(table=(0.02 * normal(V, D)).to(s["table_dtype"]), io=dt)
        else:
            s.update(dy=(1e-3 * normal(T, D)).to(dt))
        return s
    if op.startswith("block_norm"):
        rows = case["rows"]
        # a residual stream with a few strong channels, a block's output, its gate
        s.update(r=(normal(rows, D) * (0.5 + 3 * uniform(D) ** 4)).to(dt), weight=1 + 0.1 * normal(D), scale=0.5,
                 o=None, z=None, post_weight=None)
        if case["block"]:
            s.update(o=(normal(rows, D) * (0.2 + uniform(D))).to(dt), post_weight=1 + 0.1 * normal(D))
        if case["gate"]:
            s["z"] = normal(rows, D).to(dt)
        if op == "block_norm_bwd":
            f = _plain_block_norm(s)
            s.update(r_out=f["r_out"], rstd=f["rstd"], post_rstd=f.get("post_rstd"), dy=normal(rows, D).to(dt),
                     dr_out=normal(rows, D).to(dt))
            del s["r"]
        return s
    T, V = case["T"], case["V"]
    w = normal(V, D) * D ** -0.5
    targets = (V ** uniform(T).double()).long().sub(1).clamp(0, V - 1)
    # final-norm activations that favour their target by up to ten: from lost to nearly certain tokens
    x = normal(T, D) + 10 * uniform(T, 1) * w[targets]
    targets = torch.where(uniform(T) < case["ignored"], -100, targets)
    s.update(x=x.to(dt), weight=w.to(dt), targets=targets, scale=1.0)
    if op == "xent_bwd":
        s["lse"] = _plain_xent(s)["lse"]
        count = max(1, round(T * (1 - case["ignored"])))
        s["dloss"] = torch.full((T,), 1 / count, device=DEVICE)  # the mean over the tokens that count
        s["dlse"] = 2e-4 / count * s["lse"] if case["penalty"] else None  # of 1e-4 mean lse^2
    return s


# ---- the plain forms -----------------------------------------------------------------------

def _rms(x):
    rstd = torch.rsqrt(x.square().mean(1) + EPS)
    return x * rstd[:, None], rstd


def _plain_block_norm(s):
    io = s["r"].dtype
    got = {}
    r = s["r"].float()
    if s["o"] is not None:
        a, post_rstd = _rms(s["o"].float())
        a = a * s["post_weight"]
        if s["z"] is not None:
            z = s["z"].float()
            a = a * (z * torch.sigmoid(z))
        got = {"r_out": (r + s["scale"] * a).to(io), "post_rstd": post_rstd}
    else:
        got = {"r_out": s["r"]}
    xh, rstd = _rms(got["r_out"].float())
    return {"y": (xh * s["weight"]).to(io), "rstd": rstd, **got}


def _plain_block_norm_bwd(s):
    io = s["dy"].dtype
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    rh = s["r_out"].float() * rstd
    u = dy * s["weight"]
    G = s["dr_out"].float() + rstd * (u - rh * (u * rh).mean(1, keepdim=True))
    got = {"dr": G.to(io), "dweight": (dy * rh).sum(0)}
    if s["o"] is not None:
        prstd = s["post_rstd"][:, None]
        oh = s["o"].float() * prstd
        da = s["scale"] * G
        if s["z"] is not None:
            z = s["z"].float()
            sig = torch.sigmoid(z)
            got["dz"] = (da * (oh * s["post_weight"]) * (sig * (1 + z * (1 - sig)))).to(io)
            da = da * (z * sig)
        u = da * s["post_weight"]
        got["do"] = (prstd * (u - oh * (u * oh).mean(1, keepdim=True))).to(io)
        got["dpost_weight"] = (da * oh).sum(0)
    return got


def _plain_xent(s):
    logits = (s["x"].float() @ s["weight"].float().t()) * s["scale"]
    t = s["targets"]
    ok = (t >= 0) & (t < logits.shape[1])
    top = logits.amax(1)
    lse = top + (logits - top[:, None]).exp().sum(1).log()
    loss = lse - logits.gather(1, t.clamp(0, logits.shape[1] - 1)[:, None])[:, 0]
    return {"loss": torch.where(ok, loss, 0.0), "lse": torch.where(ok, lse, 0.0)}


def _plain_xent_bwd(s):
    x, w, t = s["x"].float(), s["weight"].float(), s["targets"]
    ok = (t >= 0) & (t < w.shape[0])
    dloss = torch.where(ok, s["dloss"], 0.0)
    both = dloss if s["dlse"] is None else dloss + torch.where(ok, s["dlse"], 0.0)
    p = ((x @ w.t()) * s["scale"] - s["lse"][:, None]).exp()
    g = torch.where(ok[:, None], p * both[:, None], 0.0)
    g.scatter_add_(1, t.clamp(0, w.shape[0] - 1)[:, None], -dloss[:, None])
    g = g * s["scale"]
    io = s["x"].dtype
    return {"dx": (g @ w).to(io), "dweight": (g.t() @ torch.where(ok[:, None], x, 0.0)).to(io)}


def _run_plain(s):
    op = s["op"]
    if op == "embed_fwd":
        ids = s["ids"]
        ok = (ids >= 0) & (ids < s["V"])
        rows = s["table"][ids.clamp(0, s["V"] - 1)].float() * s["scale"]
        return {"y": torch.where(ok[:, None], rows, 0.0).to(s["io"])}
    if op == "embed_bwd":
        ids = s["ids"]
        ok = (ids >= 0) & (ids < s["V"])
        # one row more, which takes the positions without a token
        d = torch.zeros(s["V"] + 1, s["dy"].shape[1], device=DEVICE)
        d.index_add_(0, torch.where(ok, ids, s["V"]), s["dy"].float())
        return {"dtable": (d[: s["V"]] * s["scale"]).to(s["table_dtype"])}
    if op == "block_norm_fwd":
        return _plain_block_norm(s)
    if op == "block_norm_bwd":
        return _plain_block_norm_bwd(s)
    return _plain_xent(s) if op == "xent_fwd" else _plain_xent_bwd(s)


def _run_own(s):
    import selective_state_space_msm_amd as msm
    op = s["op"]
    if op == "embed_fwd":
        return {"y": msm.msm_embed_fwd(s["ids"], s["table"], s["scale"], io=s["io"])}
    if op == "embed_bwd":
        return {"dtable": msm.msm_embed_bwd(s["ids"], s["dy"], s["V"], s["scale"], table_dtype=s["table_dtype"])}
    if op == "block_norm_fwd":
        r_out, y, rstd, post_rstd = msm.msm_block_norm_fwd(s["r"], s["weight"], s["o"], s["post_weight"], s["z"],
                                                           s["scale"], eps=EPS, return_stats=True)
        got = {"y": y, "rstd": rstd, "r_out": r_out}
        return got if post_rstd is None else {**got, "post_rstd": post_rstd}
    if op == "block_norm_bwd":
        d = msm.msm_block_norm_bwd(s["r_out"], s["dy"], s["rstd"], s["weight"], s["o"], s["post_rstd"],
                                   s["post_weight"], s["z"], s["scale"], dr_out=s["dr_out"])
        return {n: t for n, t in d.items() if t is not None}
    if op == "xent_fwd":
        loss, lse = msm.msm_linear_cross_entropy_fwd(s["x"], s["weight"], s["targets"], s["scale"], return_lse=True)
        return {"loss": loss, "lse": lse}
    return msm.msm_linear_cross_entropy_bwd(s["x"], s["weight"], s["targets"], s["lse"], s["dloss"], s["scale"],
                                            dlse=s["dlse"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- definitions in 64 bits ------------------------------------------------------------------

def _norm64(x):
    return x / (x.pow(2).sum(1, keepdim=True) / x.shape[1] + EPS).sqrt()


def exact(case, seed):
    s = prepare(case, seed)
    op, D = s["op"], case["D"]
    w = {n: t.double() for n, t in s.items() if torch.is_tensor(t) and t.is_floating_point()}
    if op == "embed_fwd":
        y = torch.zeros(case["T"], D, dtype=torch.float64, device=DEVICE)
        at = torch.nonzero((s["ids"] >= 0) & (s["ids"] < s["V"]))[:, 0]
        y[at] = w["table"][s["ids"][at]] * s["scale"]
        return {"y": y}
    if op == "embed_bwd":
        # the sum over a token's places: differences of a running sum in the tokens' order
        order = torch.argsort(s["ids"])
        total = torch.cat([torch.zeros(1, D, dtype=torch.float64, device=DEVICE), w["dy"][order].cumsum(0)])
        ids, every = s["ids"][order], torch.arange(s["V"], device=DEVICE)
        first, last = torch.searchsorted(ids, every), torch.searchsorted(ids, every, right=True)
        return {"dtable": (total[last] - total[first]) * s["scale"]}
    if op == "block_norm_fwd":
        io, r = s["r"].dtype, w["r"]
        got = {}
        if case["block"]:
            a = _norm64(w["o"]) * w["post_weight"]
            if case["gate"]:
                a = a * w["z"] / (1 + (-w["z"]).exp())
            r = r + s["scale"] * a
            got["post_rstd"] = (w["o"].pow(2).sum(1) / D + EPS) ** -0.5
        held = r.to(io).double()
        return {"y": _norm64(held) * w["weight"], "rstd": (held.pow(2).sum(1) / D + EPS) ** -0.5,
                "r_out": r, **got}
    if op == "block_norm_bwd":
        # the norms are rebuilt from their inputs with the statistics that the forward gave
        def normed(x, rstd):  # as a function of x whose value uses rstd: d(rstd) = -rstd^3 x dx / D
            r3 = rstd[:, None] ** 3
            return x * (rstd[:, None] - r3 * ((x - x.detach()) * x.detach()).sum(1, keepdim=True) / D)

        leaf = {n: w[n].clone().requires_grad_() for n in ("weight", "post_weight", "o", "z") if n in w}
        r_in = w["r_out"].clone().requires_grad_()  # at r' itself: dr' and dr are the same
        y = normed(r_in, w["rstd"]) * leaf["weight"]
        grads = torch.autograd.grad((w["dy"] * y).sum() + (w["dr_out"] * r_in).sum(), [r_in, leaf["weight"]])
        got = {"dr": grads[0], "dweight": grads[1]}
        if case["block"]:
            a = normed(leaf["o"], w["post_rstd"]) * leaf["post_weight"]
            if case["gate"]:
                a = a * leaf["z"] * torch.sigmoid(leaf["z"])
            names = ["o", "post_weight"] + (["z"] if case["gate"] else [])
            found = torch.autograd.grad((grads[0] * s["scale"] * a).sum(), [leaf[n] for n in names])
            got.update(zip(["do", "dpost_weight", "dz"], found))
        return got
    at = torch.nonzero((s["targets"] >= 0) & (s["targets"] < case["V"]))[:, 0]
    x, t = w["x"][at], s["targets"][at]
    logits = torch.matmul(x, w["weight"].t().contiguous()).mul_(s["scale"])
    if op == "xent_fwd":
        lse = torch.logsumexp(logits, 1)
        loss = lse - (x * w["weight"][t]).sum(1) * s["scale"]

        def whole(v):
            return torch.zeros(case["T"], dtype=torch.float64, device=DEVICE).index_copy_(0, at, v)

        return {"loss": whole(loss), "lse": whole(lse)}
    g = logits.sub_(w["lse"][at, None]).exp_()
    dloss = w["dloss"][at]
    g.mul_((dloss if s["dlse"] is None else dloss + w["dlse"][at])[:, None])
    g[torch.arange(len(at), device=DEVICE), t] -= dloss
    g.mul_(s["scale"])
    dx = torch.zeros_like(w["x"]).index_copy_(0, at, torch.matmul(g, w["weight"]))
    return {"dx": dx, "dweight": torch.matmul(g.t().contiguous(), x)}


def work(case):
    """Each input read once and each output written once; operations of the definitions.  Tokens
    without a target take no part in the cross entropy's products."""
    es = 2 if case["io"] == "bf16" else 4
    op, D = case["op"], case["D"]
    if op.startswith("embed"):
        T, V, ts = case["T"], case["V"], 2 if case["table"] == "bf16" else 4
        if op == "embed_fwd":
            return {"bytes": 8 * T + min(T, V) * D * ts + T * D * es, "flops": T * D}
        return {"bytes": 8 * T + T * D * es + V * D * ts, "flops": 2 * T * D}
    if op.startswith("block_norm"):
        n, rows, block, gate = case["rows"] * case["D"], case["rows"], case["block"], case["gate"]
        stats = 4 * rows * (1 + block) + 4 * D * (1 + block)
        if op == "block_norm_fwd":
            return {"bytes": n * es * (2 + 2 * block + gate) + stats, "flops": n * (4 + 6 * block + 6 * gate)}
        return {"bytes": n * es * (4 + 2 * block + 2 * gate) + stats + 4 * D * (1 + block),
                "flops": n * (10 + 10 * block + 12 * gate)}
    T, V = case["T"], case["V"]
    products = 2 * T * (1 - case["ignored"]) * V * D
    if op == "xent_fwd":
        return {"bytes": (T * D + V * D) * es + 16 * T, "flops": products}
    return {"bytes": 2 * (T * D + V * D) * es + (24 if case["penalty"] else 20) * T, "flops": 3 * products}
