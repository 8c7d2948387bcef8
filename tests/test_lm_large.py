"""Arrays past 2^32 bytes and 2^31 elements: the far ends against small calls on the same values."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_embedding_past_32_bits():
    import selective_state_space_msm_amd as msm
    V, D = (1 << 22) + 5, 1032  # 4.3e9 elements
    table = torch.empty(V, D, dtype=BF, device="cuda")
    far = [0, 1, (1 << 21) - 1, 1 << 21, V - 2, V - 1]
    for v in far:
        table[v] = torch.randn(D, device="cuda").to(BF)
    ids = torch.tensor(far + [V, -1], device="cuda")
    y = msm.msm_embed_fwd(ids, table, 2.0)
    assert torch.equal(y[:-2], table[far] * 2) and bool((y[-2:] == 0).all())
    del table
    dy = torch.randn(5000, D, device="cuda").to(BF)
    at = torch.tensor(far, device="cuda")[torch.arange(5000, device="cuda") % len(far)]
    d = msm.msm_embed_bwd(at, dy, V)
    small = msm.msm_embed_bwd(torch.arange(5000, device="cuda") % len(far), dy, len(far))
    assert torch.equal(d[far], small)
    d[far] = 0
    assert not bool(d.view(torch.int32).any())


def test_tokens_past_32_bits():
    import selective_state_space_msm_amd as msm
    T, D = (1 << 21) + 77, 1040  # 2.2e9 elements
    table = torch.randn(40, D, device="cuda").to(BF)
    ids = torch.randint(40, (T,), device="cuda")
    y = msm.msm_embed_fwd(ids, table)
    assert torch.equal(y[-3:], table[ids[-3:]]) and torch.equal(y[1 << 21], table[ids[1 << 21]])
    y.zero_()
    y[-5:] = 1
    d = msm.msm_embed_bwd(ids, y, 40, table_dtype=torch.float32)
    assert torch.equal(d, torch.bincount(ids[-5:], minlength=40).float()[:, None].expand(40, D))


def test_block_norm_past_32_bits():
    import selective_state_space_msm_amd as msm
    rows, D = (1 << 20) + 3, 2056  # 2.2e9 elements
    r = torch.randn(1, D, device="cuda").to(BF).expand(rows, D).contiguous()
    r[-1] = torch.randn(D, device="cuda").to(BF)
    w = torch.rand(D, device="cuda")
    # the block's output and gate are the stream itself: the inputs may share memory
    r_out, y, rstd, q = msm.msm_block_norm_fwd(r, w, r, w, r, 0.5, return_stats=True)
    few = r[-2:].contiguous()
    s_out, sy, srstd, sq = msm.msm_block_norm_fwd(few, w, few, w, few, 0.5, return_stats=True)
    assert torch.equal(r_out[-2:], s_out) and torch.equal(y[-2:], sy) and torch.equal(rstd[-2:], srstd) and torch.equal(q[-2:], sq)
    assert torch.equal(y[: 1 << 20], y[:1].expand(1 << 20, D))
    d = msm.msm_block_norm_bwd(r_out, y, rstd, w, r, q, w, r, 0.5, dr_out=y)
    s = msm.msm_block_norm_bwd(s_out, sy, srstd, w, few, sq, w, few, 0.5, dr_out=sy)
    for n in ("dr", "do", "dz"):
        assert torch.equal(d[n][-2:], s[n]) and torch.equal(d[n][:1], d[n][(1 << 20) : (1 << 20) + 1]), n


@pytest.mark.parametrize("T", [7, 150])
def test_weights_past_32_bits(T):
    import selective_state_space_msm_amd as msm
    V, D = (1 << 20) + 9, 2056  # 2.2e9 elements
    w = torch.zeros(V, D, dtype=BF, device="cuda")
    x = torch.randn(T, D, device="cuda").to(BF)
    far = torch.tensor([0, 3, 1 << 20, V - 1], device="cuda")
    w[far] = 0.02 * torch.randn(4, D, device="cuda").to(BF)
    t = far[torch.arange(T, device="cuda") % 4]
    loss, lse = msm.msm_linear_cross_entropy_fwd(x, w, t, return_lse=True)
    logits = (x.double() @ w[far].double().t())
    want = torch.log((V - 4) + logits.exp().sum(1))
    assert torch.allclose(lse.double(), want, rtol=1e-6)
    assert torch.allclose(loss.double(), want - logits.gather(1, (torch.arange(T, device="cuda") % 4)[:, None])[:, 0], rtol=1e-6, atol=1e-5)
    one = torch.ones(T, device="cuda")
    d = msm.msm_linear_cross_entropy_bwd(x, w, t, lse, one)
    p = (logits - lse.double()[:, None]).exp()
    p[torch.arange(T), torch.arange(T) % 4] -= 1
    dw = p.t() @ x.double()
    # g and the result are rounded to bf16
    tol = 2.0 ** -7 * (p.abs().t() @ x.double().abs()) + 1e-6
    assert bool(((d["dweight"][far].double() - dw).abs() <= tol).all())
    other = (-lse.double()).exp() @ x.double()  # of every row of zeros
    tol = 2.0 ** -7 * ((-lse.double()).exp() @ x.double().abs())
    for v in (1, (1 << 20) - 1, V - 2):
        assert bool(((d["dweight"][v].double() - other).abs() <= tol).all()), v


@pytest.mark.parametrize("T,io", [(262147, torch.float32), (524301, torch.float32), (524301, BF)])
def test_parts_of_tokens_past_32_bits(T, io):
    """fp32 rows in three parts that lie 1.1e9 and 2.2e9 elements apart, bf16 rows of 2.2e9, most rows left out: against
    float64 on the rows that take part.  The workspaces hold NaN, so what is not written where it is read shows."""
    import selective_state_space_msm_amd as msm
    V, D = 64, 4100
    gen = torch.Generator().manual_seed(T)
    live = torch.cat([torch.randperm(T, generator=gen)[:150], torch.tensor([0, T - 1])]).unique()
    x = torch.full((T, D), float("nan"), dtype=io, device="cuda")
    x[live.cuda()] = torch.randn(len(live), D, generator=gen).to(io).cuda()
    w = (D ** -0.5 * torch.randn(V, D, generator=gen)).to(io).cuda()
    t = torch.full((T,), -100)
    t[live] = torch.randint(V, (len(live),), generator=gen)
    t, live = t.cuda(), live.cuda()
    dl = torch.randn(T, generator=gen).cuda()

    def space(size):
        return torch.full((size(T, V, D, io),), 255, dtype=torch.uint8, device="cuda")

    loss, lse = msm.msm_linear_cross_entropy_fwd(x, w, t, return_lse=True, workspace=space(msm.msm_linear_cross_entropy_fwd_workspace_bytes))
    xd, wd, at = x[live].double(), w.double(), t[live]
    logits = xd @ wd.t()
    want = torch.logsumexp(logits, 1)
    # a logit's products leave out less than 2^-20 of a term and are summed in six rounds of D terms; the terms are of
    # either sign, and their errors as well: 16 standard deviations of the sum's
    err = 16 * (6 * D) ** 0.5 * 2.0 ** -24 * (xd.square() @ wd.square().t()).sqrt().max() + 2.0 ** -20
    assert bool(((lse[live].double() - want).abs() <= err + 2.0 ** -20 * want.abs()).all())
    assert bool(((loss[live].double() - (want - logits.gather(1, at[:, None])[:, 0])).abs() <= 2 * err + 2.0 ** -19 * want.abs()).all())
    left = torch.ones(T, dtype=torch.bool, device="cuda")
    left[live] = False
    assert not bool(loss[left].any()) and not bool(lse[left].any())
    d = msm.msm_linear_cross_entropy_bwd(x, w, t, lse, dl, workspace=space(msm.msm_linear_cross_entropy_bwd_workspace_bytes))
    g = (logits - lse[live].double()[:, None]).exp() * dl[live].double()[:, None]
    g[torch.arange(len(live)), at] -= dl[live].double()
    for name, got, ref, size in (("dx", d["dx"][live], g @ wd, g.abs() @ wd.abs()), ("dweight", d["dweight"], g.t() @ xd, g.abs().t() @ xd.abs())):
        # g: its logit's error and 2^-20 of itself; the products' and the sum's 2^-20 and fewer than 64 + 152 roundings
        tol = (err + 2.0 ** -18) * size + 6 * 256 * 2.0 ** -24 * size
        if io == BF:  # g and the result are rounded to bf16
            tol = tol + 2.0 ** -7 * size
        assert bool(((got.double() - ref).abs() <= tol).all()), name
    for i in range(0, T, 65536):  # dx of the rows that are left out
        assert not bool(d["dx"][i : i + 65536][left[i : i + 65536]].any())
