"""Embedding, block norm, delta rule, cross entropy and clipping together, as the language model of examples/ uses them."""
import importlib.util
import pathlib

import pytest
import torch
import torch.nn.functional as F

import lm_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "recurrent_lm.py"
    spec = importlib.util.spec_from_file_location("recurrent_lm", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def plain(example, model):
    """The same model in float64 on the CPU, on the plain definitions."""

    class Plain(example.RecurrentLM):
        def __init__(self):
            vars(self).update(vars(model))
            self.io = torch.float64
            self.params = {n: p.detach().double().cpu().requires_grad_() for n, p in model.params.items()}

        def _heads(self, y, i):
            q, k = (F.normalize(self._linear(y, "%d.%s" % (i, n)).unflatten(-1, (self.heads, self.size)), dim=-1) for n in "qk")
            v = self._linear(y, "%d.v" % i).unflatten(-1, (self.heads, self.size))
            return q, k, v, F.logsigmoid(self._linear(y, "%d.g" % i) + 4), torch.sigmoid(self._linear(y, "%d.beta" % i))

        def losses(self, ids, targets, offsets):
            def mix(i, q, k, v, g, beta):
                out = []
                for a, b in zip(offsets.tolist()[:-1], offsets.tolist()[1:]):
                    S = torch.zeros(self.heads, self.size, self.size, dtype=torch.float64)
                    for t in range(a, b):
                        kt, qt = (z[t][:, :, None] for z in (k, q))
                        S = g[t].exp()[:, None, None] * S
                        e = v[t] - (S * kt).sum(1)
                        S = S + kt * (beta[t][:, None] * e)[:, None, :]
                        out.append(self.size ** -0.5 * (S * qt).sum(1))
                return torch.stack(out)

            def embed(ids, table, scale, io):
                ok = (ids >= 0) & (ids < table.shape[0])
                return torch.where(ok[:, None], scale * table[ids.clamp(0, table.shape[0] - 1)], 0.0)

            y = self._run(ids, mix, lambda r, w, o, pw, z, s: lm_ref.block_norm_fwd(r, w, o, pw, z, s)[:2], embed)
            loss, lse, _ = lm_ref.xent_fwd(y, self.params["head"], targets, 1.0)
            return loss, lse

    return Plain()


def mean(model, ids, targets, offsets):
    loss, lse = model.losses(ids, targets, offsets)
    return (loss + 0.01 * lse.square()).sum() / (targets >= 0).sum()


def test_gradients_of_the_model(example):
    gen = torch.Generator().manual_seed(3)
    P = example.chain(83, gen)
    model = example.RecurrentLM(83, dim=70, size=24, io=torch.float32, seed=3)
    ids, targets, offsets = example.draw(P, [40, 0, 1, 67, 2, 90], gen)
    ids[5] = -1  # padding
    ref = plain(example, model)
    loss = mean(model, ids.cuda(), targets.cuda(), offsets.cuda())
    loss.backward()
    rloss = mean(ref, ids, targets, offsets)
    rloss.backward()
    # two layers of fp32 sums of up to 200 terms, a few of them behind one another
    assert abs(loss.item() - rloss.item()) <= 1e-5 * rloss.item()
    for n, p in model.params.items():
        want = ref.params[n].grad
        err = (p.grad.double().cpu() - want).norm().item()
        assert err <= 1e-4 * want.norm().item(), (n, err)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_training_runs(example, io):
    gen = torch.Generator().manual_seed(0)
    model = example.RecurrentLM(50, io=io, seed=0)
    for loss, norm in example.train(model, example.chain(50, gen), 5, gen, sequences=6, longest=20):
        assert 0 < loss < 20 and norm > 0


@pytest.mark.parametrize("io,tol", [(torch.float32, 1e-4), (torch.bfloat16, 0.1)])
def test_serving_token_by_token(example, io, tol):
    """A prompt's states and the steps from them give what the whole pass gives: fp32 to its sums, bf16 to
    the roundings (2^-8 each at most) of two layers' activations."""
    gen = torch.Generator().manual_seed(5)
    P = example.chain(40, gen)
    model = example.RecurrentLM(40, io=io, seed=5)
    ids = example.draw(P, [60] * 9, gen)[0].view(9, 60).cuda()
    whole, _ = model.prefill(ids)
    y, states = model.prefill(ids[:, :45].contiguous())
    y = y[:, -1].contiguous()
    for t in range(45, 60):
        want = whole[:, t - 1]
        assert (y.float() - want.float()).norm() <= tol * want.float().norm()
        logits = want.float() @ model.params["head"].to(io).float().t()
        lp = torch.log_softmax(logits, 1).gather(1, ids[:, t : t + 1])[:, 0]
        assert (model.log_prob(y, ids[:, t].contiguous()) - lp).norm() <= tol * lp.norm()
        y = model.step(ids[:, t].contiguous(), states)
