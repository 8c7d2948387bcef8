"""The block operators on arrays past 2^32 bytes and 2^31 elements: the last part of a large call
against the same part by itself, which takes the same sums in the same order."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def rnd(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def gen():
    return torch.Generator("cuda").manual_seed(70)


def room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip("needs %d GiB" % gigabytes)


@pytest.mark.parametrize("packed", [False, True])
def test_delta_rule(packed):
    import selective_state_space_msm_amd as msm
    room(100)
    r = gen()
    Bt, L, Hk, H, K, V = 5, 60001, 8, 32, 64, 256  # v: 4.9 GB
    lead = (Bt * L,) if packed else (Bt, L)
    unit = lambda x: torch.nn.functional.normalize(x.float(), dim=-1).bfloat16()
    q, k, v, do = unit(rnd(r, *lead, Hk, K)), unit(rnd(r, *lead, Hk, K)), rnd(r, *lead, H, V), rnd(r, *lead, H, V)
    g = -0.1 * rnd(r, *lead, H, dtype=torch.float32).square()
    beta = torch.sigmoid(rnd(r, *lead, H, dtype=torch.float32))
    where, last = {}, {}
    part = lambda t: t[-1:]
    if packed:
        where["seq_offsets"] = torch.arange(Bt + 1, dtype=torch.int32, device="cuda") * L
        last["seq_offsets"] = where["seq_offsets"][:2]
        part = lambda t: t[-L:]
    assert v.numel() * 2 > 1 << 32
    ins = (q, k, v, g, beta)
    mine = tuple(part(t).clone() for t in ins)
    o, S = msm.msm_delta_rule_fwd(*ins, return_last_state=True, **where)
    wo, wS = msm.msm_delta_rule_fwd(*mine, return_last_state=True, **last)
    assert torch.equal(part(o), wo) and torch.equal(S[-1:], wS)
    del o, S
    d = msm.msm_delta_rule_bwd(*ins, do, **where)
    want = msm.msm_delta_rule_bwd(*mine, part(do).clone(), **last)
    for n in want:
        assert torch.equal(part(d[n]), want[n]), n


def test_delta_rule_step():
    import selective_state_space_msm_amd as msm
    room(20)
    r = gen()
    Bt, Hk, H, K, V = 600, 8, 32, 256, 256  # states: 5 GB
    q, k, v = rnd(r, Bt, Hk, K), rnd(r, Bt, Hk, K) / 16, rnd(r, Bt, H, V)
    g, beta = -rnd(r, Bt, H, dtype=torch.float32).square(), torch.rand(Bt, H, generator=r, device="cuda")
    S = rnd(r, Bt, H, K, V, dtype=torch.float32)
    mine = tuple(t[-16:].clone() for t in (q, k, v, g, beta, S))
    o = msm.msm_delta_rule_step(q, k, v, g, beta, S)
    assert torch.equal(o[-16:], msm.msm_delta_rule_step(*mine)) and torch.equal(S[-16:], mine[-1])


@pytest.mark.parametrize("rows,D", [(270000, 8192), (430000, 5001)])
def test_layer_norm(rows, D):
    import selective_state_space_msm_amd as msm
    room(40)
    r = gen()
    x, dy = rnd(r, rows, D), rnd(r, rows, D)
    assert x.numel() > 1 << 31
    w, b = rnd(r, D, dtype=torch.float32), rnd(r, D, dtype=torch.float32)
    y, mean, rstd = msm.msm_layer_norm_fwd(x, w, b, return_stats=True)
    mine = x[-500:].clone()
    wy, wmean, wrstd = msm.msm_layer_norm_fwd(mine, w, b, return_stats=True)
    assert torch.equal(y[-500:], wy) and torch.equal(mean[-500:], wmean) and torch.equal(rstd[-500:], wrstd)
    del y
    d = msm.msm_layer_norm_bwd(x, dy, mean, rstd, w, bias_grad=True)
    want = msm.msm_layer_norm_bwd(mine, dy[-500:].clone(), wmean, wrstd, w)
    assert torch.equal(d["dx"][-500:], want["dx"])
    total = dy.sum(0, dtype=torch.float64)
    # sqrt(rows) roundings of 2^-24 of partial sums the size of the result and below
    assert float((d["dbias"] - total).norm()) <= 2.0 ** -24 * rows ** 0.5 * float(total.norm())


@pytest.mark.parametrize("offset", [0, 1])
def test_clipping(offset):
    import selective_state_space_msm_amd as msm
    room(40)
    n = (1 << 31) + 12345
    x = torch.ones(n + offset, dtype=torch.bfloat16, device="cuda")[offset:]
    x[-3:] = 512.0
    out = torch.zeros(n + offset, dtype=torch.bfloat16, device="cuda")[offset:]
    want = float(n - 3 + 3 * 512 ** 2) ** 0.5
    norm = msm.msm_grad_clip([x], 0.5 * want, eps=0.0, out=[out])
    assert abs(float(norm) - want) <= 1e-7 * want
    # 0.5 to two fp32 roundings, which bf16 rounds away
    assert bool((out[:-3] == 0.5).all()) and bool((out[-3:] == 256.0).all())
