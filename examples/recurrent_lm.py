"""A small language model out of this library's operators: trained on packed sequences, then served.

Tokens come from a random Markov chain, so the loss has a floor that the chain's entropy sets.  The
stream from ids to loss is made of the library's operators and plain products with the weights:

  training  msm_embed_fwd -> [msm_block_norm_fwd -> msm_delta_rule_fwd] x layers ->
            msm_block_norm_fwd -> msm_linear_cross_entropy_fwd, their gradients, msm_grad_clip
  serving   a prompt through the same with the delta rule's states kept, then one token at a time:
            msm_embed_fwd, msm_block_norm_fwd with the stream updated in place, msm_delta_rule_step,
            and msm_linear_cross_entropy_fwd for a token's log-probability

A block's output o is normed, gated and added to the stream r by the next block's
msm_block_norm_fwd, which also norms the sum for that block: r <- r + scale pw RMS(o) silu(z).

    python examples/recurrent_lm.py --steps 200
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import selective_state_space_msm_amd as msm  # noqa: E402


class Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale, io):
        ctx.save_for_backward(ids)
        ctx.of = table.shape[0], table.dtype, scale
        return msm.msm_embed_fwd(ids, table, scale, io=io)

    @staticmethod
    def backward(ctx, dy):
        V, dtype, scale = ctx.of
        return None, msm.msm_embed_bwd(ctx.saved_tensors[0], dy.contiguous(), V, scale, table_dtype=dtype), None, None


class BlockNorm(torch.autograd.Function):
    """(r_out, y) of msm_block_norm_fwd; o, post_weight and z may be None."""

    @staticmethod
    def forward(ctx, r, weight, o, post_weight, z, scale):
        r_out, y, rstd, post_rstd = msm.msm_block_norm_fwd(r, weight, o, post_weight, z, scale, return_stats=True)
        ctx.save_for_backward(r_out, rstd, weight, o, post_rstd, post_weight, z)
        ctx.scale = scale
        return (r.view_as(r) if o is None else r_out), y

    @staticmethod
    def backward(ctx, dr_out, dy):
        r_out, rstd, weight, o, post_rstd, post_weight, z = ctx.saved_tensors
        d = msm.msm_block_norm_bwd(r_out, dy.contiguous(), rstd, weight, o, post_rstd, post_weight, z, ctx.scale,
                                   dr_out=dr_out.contiguous())
        return d["dr"], d["dweight"], d["do"], d["dpost_weight"], d["dz"], None


class DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, seq_offsets):
        ctx.save_for_backward(q, k, v, g, beta, seq_offsets)
        return msm.msm_delta_rule_fwd(q, k, v, g, beta, seq_offsets=seq_offsets)

    @staticmethod
    def backward(ctx, do):
        q, k, v, g, beta, seq_offsets = ctx.saved_tensors
        d = msm.msm_delta_rule_bwd(q, k, v, g, beta, do.contiguous(), seq_offsets=seq_offsets)
        return d["dq"], d["dk"], d["dv"], d["dg"], d["dbeta"], None


class CrossEntropy(torch.autograd.Function):
    """Loss of every row, and lse."""

    @staticmethod
    def forward(ctx, x, weight, targets):
        loss, lse = msm.msm_linear_cross_entropy_fwd(x, weight, targets, return_lse=True)
        ctx.save_for_backward(x, weight, targets, lse)
        return loss, lse

    @staticmethod
    def backward(ctx, dloss, dlse):
        x, weight, targets, lse = ctx.saved_tensors
        d = msm.msm_linear_cross_entropy_bwd(x, weight, targets, lse, dloss.contiguous(), dlse=dlse.contiguous())
        return d["dx"], d["dweight"], None


class RecurrentLM:
    """Parameters are float32, the operators' inputs `io` (bfloat16 or float32)."""

    def __init__(self, vocab, dim=96, heads=3, size=32, layers=2, io=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=gen)
        self.vocab, self.heads, self.size, self.layers, self.io = vocab, heads, size, layers, io
        self.scale = (2 * layers) ** -0.5  # of a block's part of the stream
        p = {"embed": rnd(vocab, dim) * dim ** -0.5, "head": rnd(vocab, dim) * dim ** -0.5}
        for i in range(layers + 1):
            p["%d.norm" % i] = torch.ones(dim)
        for i in range(layers):
            p["%d.post" % i] = torch.ones(dim)
            for name, n in (("q", heads * size), ("k", heads * size), ("v", heads * size), ("g", heads), ("beta", heads), ("z", dim)):
                p["%d.%s" % (i, name)] = rnd(n, dim) * dim ** -0.5
            p["%d.o" % i] = rnd(dim, heads * size) * (heads * size) ** -0.5
        self.params = {n: t.to(device).requires_grad_() for n, t in p.items()}
        self.embed_scale = dim ** 0.5

    def _linear(self, x, name):
        return F.linear(x, self.params[name].to(x.dtype))

    def _heads(self, y, i):
        q, k = (F.normalize(self._linear(y, "%d.%s" % (i, n)).float().unflatten(-1, (self.heads, self.size)), dim=-1).to(self.io)
                for n in "qk")
        v = self._linear(y, "%d.v" % i).unflatten(-1, (self.heads, self.size))
        g = F.logsigmoid(self._linear(y, "%d.g" % i).float() + 4)
        return q, k, v, g, torch.sigmoid(self._linear(y, "%d.beta" % i).float())

    def _run(self, ids, mix, norm, embed):
        """The last norm's output; mix(layer, q, k, v, g, beta) is the delta rule."""
        r, o, z, post = embed(ids, self.params["embed"], self.embed_scale, self.io), None, None, None
        for i in range(self.layers):
            r, y = norm(r, self.params["%d.norm" % i], o, post, z, self.scale)
            o = self._linear(mix(i, *self._heads(y, i)).flatten(-2), "%d.o" % i)
            z, post = self._linear(y, "%d.z" % i), self.params["%d.post" % i]
        return norm(r, self.params["%d.norm" % self.layers], o, post, z, self.scale)[1]

    def losses(self, ids, targets, seq_offsets):
        """Loss and lse of every token of packed sequences, for training."""
        y = self._run(ids, lambda i, *a: DeltaRule.apply(*a, seq_offsets), BlockNorm.apply, Embed.apply)
        return CrossEntropy.apply(y, self.params["head"].to(self.io), targets)

    def _serve(self, ids, mix):
        def norm(r, w, o, post, z, scale):  # the stream is nobody else's: updated in place
            return msm.msm_block_norm_fwd(r, w, o, post, z, scale, r_out=r)

        return self._run(ids, mix, norm, lambda ids, table, scale, io: msm.msm_embed_fwd(ids, table, scale, io=io))

    @torch.no_grad()
    def prefill(self, ids):
        """Output (Bt, L, dim) of prompts and the state of every layer after them."""
        states = []

        def mix(i, *a):
            o, S = msm.msm_delta_rule_fwd(*a, return_last_state=True)
            states.append(S)
            return o

        return self._serve(ids, mix), states

    @torch.no_grad()
    def step(self, ids, states):
        """Output (Bt, dim) of one token per sequence; the states are updated in place."""
        return self._serve(ids, lambda i, *a: msm.msm_delta_rule_step(*a, states[i]))

    @torch.no_grad()
    def log_prob(self, y, ids):
        """Log-probabilities of the tokens ids that follow outputs y."""
        return -msm.msm_linear_cross_entropy_fwd(y, self.params["head"].to(self.io), ids)


def chain(vocab, gen):
    """Transition probabilities of a random Markov chain with a few likely successors a token."""
    return torch.softmax(3 * torch.randn(vocab, vocab, generator=gen), 1)


def draw(P, lengths, gen):
    """Packed tokens of walks through the chain, their successors (-100 behind a walk's end), offsets."""
    tokens, targets = [], []
    for n in lengths:
        at = torch.randint(len(P), (), generator=gen).item()
        walk = [at]
        for _ in range(n):
            at = torch.multinomial(P[at], 1, generator=gen).item()
            walk.append(at)
        tokens += walk[:n]
        targets += walk[1:n] + [-100] if n else []
    offsets = torch.tensor([0] + list(lengths)).cumsum(0).to(torch.int32)
    return torch.tensor(tokens), torch.tensor(targets), offsets


def train(model, P, steps, gen, lr=3e-3, max_norm=1.0, sequences=16, longest=64, penalty=1e-4):
    """Yields (loss, gradient norm before clipping) for every step."""
    params = list(model.params.values())
    optimiser = torch.optim.AdamW(params, lr=lr, weight_decay=0.0)
    dev = params[0].device
    for _ in range(steps):
        lengths = torch.randint(0, longest + 1, (sequences,), generator=gen).tolist()
        lengths[0] = longest
        ids, targets, offsets = (t.to(dev) for t in draw(P, lengths, gen))
        loss, lse = model.losses(ids, targets, offsets)
        count = (targets >= 0).sum()
        mean = loss.sum() / count
        optimiser.zero_grad(set_to_none=True)
        (mean + penalty * lse.square().sum() / count).backward()
        norm = msm.msm_grad_clip([p.grad for p in params], max_norm)
        optimiser.step()
        yield mean.item(), norm.item()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--vocab", type=int, default=500)
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--io", choices=("bf16", "f32"), default="bf16")
    args = ap.parse_args()
    gen = torch.Generator().manual_seed(args.seed)
    P = chain(args.vocab, gen)
    model = RecurrentLM(args.vocab, seed=args.seed, io=torch.bfloat16 if args.io == "bf16" else torch.float32)
    for i, (loss, norm) in enumerate(train(model, P, args.steps, gen)):
        if i % 20 == 0 or i + 1 == args.steps:
            print("step %4d  loss %.4f  gradient norm %.3f" % (i, loss, norm), flush=True)
    print("entropy of the chain %.4f" % -(P * P.log()).sum(1).mean().item())
    Bt, L = 32, 48
    ids, _, _ = draw(P, [L] * Bt, gen)
    ids = ids.view(Bt, L).cuda()
    half = L // 2
    whole, _ = model.prefill(ids)
    y, states = model.prefill(ids[:, :half].contiguous())
    y, worst = y[:, -1].contiguous(), 0.0
    for t in range(half, L):
        now = ids[:, t].contiguous()
        served, at_once = model.log_prob(y, now), model.log_prob(whole[:, t - 1].contiguous(), now)
        worst = max(worst, (served - at_once).abs().max().item())
        y = model.step(now, states)
    print("served token by token: log-probabilities within %.2g of the whole pass" % worst)


if __name__ == "__main__":
    main()
