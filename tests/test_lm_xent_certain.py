"""The linear cross entropy's loss of tokens that are nearly certain: the difference of two large numbers."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(5, 300), (30, 4000), (200, 300), (700, 3000), (2000, 9000)])
def test_nearly_certain_tokens(io, T, V):
    import selective_state_space_msm_amd as msm
    D, scale = 64, 0.9
    gen = torch.Generator().manual_seed(T + V)
    # a row picks one column of the weights, so that the products are exact: the target's is 512, the others' at
    # most 494 and whole, and the scaled logits 16.2 and more apart
    w = torch.randint(0, 248, (V, D), generator=gen).float() * 2
    t = torch.randint(V, (T,), generator=gen)
    column = torch.arange(T) % D
    for c in range(D):  # one word a column, the target of its rows
        v = int(t[c]) if c < T else 0
        w[v, c] = 512
        t[column == c] = v
    x = torch.zeros(T, D)
    x[torch.arange(T), column] = 1
    loss, lse = (a.cpu().double() for a in msm.msm_linear_cross_entropy_fwd(x.to(DT[io]).cuda(), w.to(DT[io]).cuda(), t.cuda(), scale, return_lse=True))
    s = float(torch.tensor(scale))
    logits = s * (x.double() @ w.double().t())
    assert float(logits.gather(1, t[:, None]).min()) > 460
    want = torch.logsumexp(logits, 1) - logits.gather(1, t[:, None])[:, 0]
    # the largest logit is the target's, and is taken from itself; the others' exponents are off by two roundings of
    # 461 log2(e), 2^-14 of a factor in all; a sum of at most 64 terms one after another and its joins, near 1
    tol = 2.0 ** -14 * want + 80 * 2.0 ** -24
    assert bool((loss >= 0).all())
    assert bool(((loss - want).abs() <= tol).all()), float((loss - want).abs().max())
    assert bool(((lse - torch.logsumexp(logits, 1)).abs() <= 4 * 2.0 ** -24 * 461 + tol).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 20, 300, 700])
def test_one_word(io, T):
    import selective_state_space_msm_amd as msm
    gen = torch.Generator().manual_seed(T)
    x, w = torch.randn(T, 200, generator=gen).to(DT[io]).cuda(), torch.randn(1, 200, generator=gen).to(DT[io]).cuda()
    loss = msm.msm_linear_cross_entropy_fwd(x, w, torch.zeros(T, dtype=torch.int64, device="cuda"), 1.7)
    assert bool((loss == 0).all())
