"""The block operators together: a small recall model trained with them, then served token by token.

A sequence is a ragged run of notes "key c has value u" (a later note on the same key replaces the
earlier one) and questions "what is the value of key c?".  The model is an embedding, `layers`
blocks  x + Wo delta_rule(layer_norm(x))  and a layer norm before the output, and every step of it
that is not a plain matrix product with the weights is one of this library's operators:

  training  packed sequences -> msm_layer_norm_fwd -> msm_delta_rule_fwd ... -> loss ->
            msm_delta_rule_bwd, msm_layer_norm_bwd -> msm_grad_clip -> AdamW
  serving   a prompt through msm_delta_rule_fwd with its last state kept, then one token at a time
            through msm_delta_rule_step on that state

    python examples/delta_block.py --steps 200
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import selective_state_space_msm_amd as msm  # noqa: E402


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        y, mean, rstd = msm.msm_layer_norm_fwd(x, weight, bias, return_stats=True)
        ctx.save_for_backward(x, mean, rstd, weight)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, mean, rstd, weight = ctx.saved_tensors
        d = msm.msm_layer_norm_bwd(x, dy.contiguous(), mean, rstd, weight, bias_grad=True)
        return d["dx"], d["dweight"], d["dbias"]


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


class RecallModel:
    """Parameters are float32, the operators' inputs `io` (bfloat16 or float32)."""

    def __init__(self, keys, values, dim=128, key_heads=2, heads=4, size=32, layers=2,
                 io=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.keys, self.values, self.io, self.layers = keys, values, io, layers
        self.key_heads, self.heads, self.size = key_heads, heads, size
        p = {"embed": torch.randn(keys * values + keys, dim, generator=gen)}

        def norm(name):
            p[name + ".weight"] = torch.ones(dim)
            p[name + ".bias"] = torch.zeros(dim)

        for i in range(layers):
            norm("%d.norm" % i)
            for name, n in (("q", key_heads * size), ("k", key_heads * size), ("v", heads * size),
                            ("g", heads), ("beta", heads)):
                p["%d.%s" % (i, name)] = torch.randn(n, dim, generator=gen) * dim ** -0.5
            p["%d.o" % i] = torch.randn(dim, heads * size, generator=gen) * (heads * size) ** -0.5
        norm("norm")
        p["out"] = torch.randn(values, dim, generator=gen) * dim ** -0.5
        self.params = {n: t.to(device).requires_grad_() for n, t in p.items()}

    def _linear(self, x, name):
        return F.linear(x, self.params[name].to(x.dtype))

    def _norm(self, x, name):
        return LayerNorm.apply(x, self.params[name + ".weight"], self.params[name + ".bias"])

    def _heads(self, x, i):
        """The delta rule's inputs for tokens x (..., dim): unit keys and queries, log decays, and
        write strengths in (0, 1)."""
        q, k = (F.normalize(self._linear(x, "%d.%s" % (i, n)).float()
                            .unflatten(-1, (self.key_heads, self.size)), dim=-1).to(self.io)
                for n in "qk")
        v = self._linear(x, "%d.v" % i).unflatten(-1, (self.heads, self.size))
        # about one part in 50 forgotten a token at first
        g = F.logsigmoid(self._linear(x, "%d.g" % i).float() + 4)
        return q, k, v, g, torch.sigmoid(self._linear(x, "%d.beta" % i).float())

    def _run(self, tokens, mix):
        """Logits; mix(layer, q, k, v, g, beta) is the delta rule."""
        x = F.embedding(tokens, self.params["embed"]).to(self.io)
        for i in range(self.layers):
            o = mix(i, *self._heads(self._norm(x, "%d.norm" % i), i))
            x = x + self._linear(o.flatten(-2), "%d.o" % i)
        return self._linear(self._norm(x, "norm"), "out").float()

    def packed(self, tokens, seq_offsets):
        """Logits (tokens, values) of packed sequences, for training."""
        return self._run(tokens, lambda i, *a: DeltaRule.apply(*a, seq_offsets))

    @torch.no_grad()
    def prefill(self, tokens):
        """Logits (Bt, L, values) of prompts and the state of every layer after them."""
        states = []

        def mix(i, *a):
            o, S = msm.msm_delta_rule_fwd(*a, return_last_state=True)
            states.append(S)
            return o

        return self._run(tokens, mix), states

    @torch.no_grad()
    def step(self, tokens, states):
        """Logits (Bt, values) of one token per sequence; the states are updated in place."""
        return self._run(tokens, lambda i, *a: msm.msm_delta_rule_step(*a, states[i]))


def draw(keys, values, lengths, gen):
    """Packed tokens, their answers (-100 where nothing is asked) and the sequences' offsets.
    A sequence of n tokens is notes in its first half and questions on noted keys after it."""
    tokens, answers = [], []
    for n in lengths:
        known = {}
        for t in range(n):
            if t < (n + 1) // 2:
                key, value = torch.randint(keys, (), generator=gen).item(), torch.randint(values, (), generator=gen).item()
                known[key] = value
                tokens.append(key * values + value)
                answers.append(-100)
            else:
                key = sorted(known)[torch.randint(len(known), (), generator=gen).item()]
                tokens.append(keys * values + key)
                answers.append(known[key])
    offsets = torch.tensor([0] + list(lengths)).cumsum(0)
    return torch.tensor(tokens), torch.tensor(answers), offsets.to(torch.int32)


def train(model, steps, gen, lr=3e-3, max_norm=1.0, sequences=32, longest=96):
    """Yields (loss, gradient norm before clipping, share of right answers) for every step."""
    params = list(model.params.values())
    optimiser = torch.optim.AdamW(params, lr=lr, weight_decay=0.0)
    dev = params[0].device
    for _ in range(steps):
        lengths = torch.randint(0, longest + 1, (sequences,), generator=gen).tolist()
        lengths[0] = longest
        tokens, answers, offsets = (t.to(dev) for t in draw(model.keys, model.values, lengths, gen))
        logits = model.packed(tokens, offsets)
        loss = F.cross_entropy(logits, answers)
        optimiser.zero_grad(set_to_none=True)
        loss.backward()
        norm = msm.msm_grad_clip([p.grad for p in params], max_norm)
        optimiser.step()
        asked = answers >= 0
        right = (logits.argmax(-1) == answers)[asked].float().mean()
        yield loss.item(), norm.item(), right.item()


def serve(model, prompts, questions):
    """Prefills prompts (Bt, L), then asks questions (Bt, n) one token at a time: logits
    (Bt, n, values)."""
    _, states = model.prefill(prompts)
    return torch.stack([model.step(t.contiguous(), states) for t in questions.unbind(1)], dim=1)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--keys", type=int, default=8)
    ap.add_argument("--values", type=int, default=8)
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--io", choices=("bf16", "f32"), default="bf16")
    args = ap.parse_args()
    gen = torch.Generator().manual_seed(args.seed)
    model = RecallModel(args.keys, args.values, seed=args.seed,
                        io=torch.bfloat16 if args.io == "bf16" else torch.float32)
    for i, (loss, norm, right) in enumerate(train(model, args.steps, gen)):
        if i % 20 == 0 or i + 1 == args.steps:
            print("step %4d  loss %.4f  gradient norm %.3f  right %.3f" % (i, loss, norm, right), flush=True)
    Bt, L = 64, 96
    tokens, answers, _ = (t.cuda() for t in draw(args.keys, args.values, [L] * Bt, gen))
    tokens, answers = tokens.view(Bt, L), answers.view(Bt, L)
    half = L // 2
    logits = serve(model, tokens[:, :half].contiguous(), tokens[:, half:])
    whole, _ = model.prefill(tokens)
    print("served token by token: right %.3f, logits within %.2g of the whole pass" % (
        (logits.argmax(-1) == answers[:, half:]).float().mean().item(),
        (logits - whole[:, half:]).abs().max().item()))


if __name__ == "__main__":
    main()
