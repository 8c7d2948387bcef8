"""The linear cross entropy where logits are infinite: by the definition, as far as that has a value."""
import pytest
import torch

pytestmark = pytest.mark.gpu
INF = float("inf")


def rows(T, V=300, D=64):
    gen = torch.Generator().manual_seed(T)
    x = (torch.rand(T, D, generator=gen) + 0.1).bfloat16().cuda()
    w = torch.randn(V, D, generator=gen).bfloat16().cuda()
    return x, w, torch.randint(V, (T,), generator=gen).cuda()


# 8 and 20: the kernel for few rows; 300: rows in their places; 700: gathered rows
@pytest.mark.parametrize("T", [8, 20, 300, 700])
@pytest.mark.parametrize("word", [0, 17, 299])
def test_a_word_of_infinite_logits(T, word):
    import selective_state_space_msm_amd as msm
    x, w, t = rows(T)
    w[word] = INF  # the rows are positive: a logit of plus infinity each
    t[0] = word
    loss, lse = msm.msm_linear_cross_entropy_fwd(x, w, t, return_lse=True)
    assert bool((lse == INF).all())
    there = t == word  # infinity minus infinity has no value
    assert bool((loss[~there] == INF).all()) and bool(torch.isnan(loss[there]).all())


@pytest.mark.parametrize("T", [8, 300, 700])
def test_one_row_of_infinite_logits(T):
    """A logit past the largest number in one row alone: the others are as they were."""
    import selective_state_space_msm_amd as msm
    x, w, t = rows(T)
    x[3] = 3e38
    w *= 1e-3  # sums of 64 terms of up to 4e-3 x 3e38: no partial sum of row 3 is past 3.4e38 but word 5's
    w[5] = 2.0
    l0, e0 = msm.msm_linear_cross_entropy_fwd(torch.cat([x[:3], x[4:]]), w, torch.cat([t[:3], t[4:]]), return_lse=True)
    l1, e1 = msm.msm_linear_cross_entropy_fwd(x, w, t, return_lse=True)
    size = x[3].double() @ w.double().abs().t()
    assert bool((size > 3.4e38).nonzero().flatten().tolist() == [5])
    assert float(e1[3]) == INF
    rest = torch.arange(T, device="cuda") != 3
    assert torch.allclose(e1[rest], e0, rtol=1e-6) and torch.allclose(l1[rest], l0, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("T", [8, 300, 700])
def test_all_logits_minus_infinity(T):
    import selective_state_space_msm_amd as msm
    x, w, t = rows(T)
    w[:] = -INF
    loss, lse = msm.msm_linear_cross_entropy_fwd(x, w, t, return_lse=True)
    assert bool((lse == -INF).all()) and bool(torch.isnan(loss).all())


@pytest.mark.parametrize("T", [8, 300, 700])
def test_nan_beside_infinity(T):
    import selective_state_space_msm_amd as msm
    x, w, t = rows(T)
    w[7], w[40] = INF, float("nan")
    loss, lse = msm.msm_linear_cross_entropy_fwd(x, w, t, return_lse=True)
    assert bool(torch.isnan(lse).all()) and bool(torch.isnan(loss).all())
