"""Token embedding and its gradient on the GPU against float64."""
import pytest
import torch

import lm_ref
from gpu_util import log

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def half(dt):
    return torch.finfo(dt).eps / 2


def device(t, offset=0):
    buf = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
    v = buf[offset:].view(t.shape)
    v.copy_(t)
    return v


def make(kind, T, V, gen):
    if kind == "one":
        return torch.full((T,), V // 2)
    if kind == "two":
        return torch.where(torch.rand(T, generator=gen) < 0.5, 0, V - 1)
    ids = (float(V) ** torch.rand(T, generator=gen, dtype=torch.float64)).long() - 1  # log-uniform
    ids = ids.clamp(0, V - 1)
    off = torch.rand(T, generator=gen)
    ids[off < 0.06] = -1
    ids[(off >= 0.06) & (off < 0.1)] = V
    ids[(off >= 0.1) & (off < 0.12)] = -(1 << 40)
    return ids


def check(T, V, D, table="f32", io="f32", kind="zipf", offset=0, scale=1.7):
    import selective_state_space_msm_amd as msm
    gen = torch.Generator().manual_seed(T * 7 + V + D)
    ids = make(kind, T, V, gen)
    log("T=%d V=%d D=%d %s %s %s" % (T, V, D, table, io, kind))
    tab = torch.randn(V, D, generator=gen).to(DT[table])
    y = msm.msm_embed_fwd(ids.cuda(), device(tab, offset), scale, io=DT[io])
    want = lm_ref.embed_fwd(ids, tab.double(), float(torch.tensor(scale)))
    # the product's rounding in fp32 and the result's
    tol = (2.0 ** -24 + half(DT[io])) * 1.01 * want.abs()
    assert bool(((y.double().cpu() - want).abs() <= tol).all())
    dy = torch.randn(T, D, generator=gen).to(DT[io])
    d = msm.msm_embed_bwd(ids.cuda(), device(dy, offset), V, scale, table_dtype=DT[table])
    want, size, n = lm_ref.embed_bwd(ids, dy.double(), V, float(torch.tensor(scale)))
    # a sum of n terms has n roundings of at most the sum of sizes, the scaling one, the result one
    tol = 1.01 * ((n + 1) * 2.0 ** -24 * size + half(DT[table]) * want.abs())
    assert bool(((d.double().cpu() - want).abs() <= tol).all())
    return d


@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 5, 16), (2, 3, 7), (63, 10, 33), (64, 100, 8), (65, 17, 129),
                                   (1000, 300, 20), (2047, 1003, 129), (4096, 513, 40), (4097, 513, 40), (5000, 70000, 9),
                                   (20000, 262145, 5), (70000, 1000, 24)])
def test_sizes(T, V, D):
    check(T, V, D)
    check(T, V, D, "bf16", "bf16")


@pytest.mark.parametrize("table,io", [("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("D", [1, 3, 8, 17, 64])
def test_mixed_types(table, io, D):
    check(300, 50, D, table, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["one", "two"])
@pytest.mark.parametrize("T", [64, 100, 1023, 3000, 40000])
def test_frequent_tokens(kind, T, io):
    check(T, 300, 40, io, io, kind)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_unaligned(io):
    check(500, 90, 129, io, io, offset=1)
    check(500, 90, 128, io, io, offset=3)


def test_sums_do_not_drift():
    """2^20 places of one token with equal gradients: a running fp32 sum would be off by 1e-3."""
    import selective_state_space_msm_amd as msm
    T = 1 << 20
    ids = torch.zeros(T, dtype=torch.int64, device="cuda")
    dy = torch.full((T, 4), 1.1, device="cuda")
    d = msm.msm_embed_bwd(ids, dy, 3)
    want = T * dy[0].double()
    # two sums of 32 (32 roundings each at most) and the last rounding
    assert bool(((d[0].double() - want).abs() <= 66 * 2.0 ** -24 * want).all())
    assert bool((d[1:] == 0).all())


def test_nothing_to_learn():
    import selective_state_space_msm_amd as msm
    ids = torch.full((5000,), -100, device="cuda")
    dy = torch.full((5000, 24), float("nan"), device="cuda")
    out = torch.full((77, 24), float("nan"), device="cuda")
    assert bool((msm.msm_embed_bwd(ids, dy, 77, dtable=out) == 0).all())
    assert bool((msm.msm_embed_fwd(ids, out + float("nan")) == 0).all())


def test_nan_stays_in_its_row():
    import selective_state_space_msm_amd as msm
    ids = torch.tensor([3, 1, 3, 0, -1], device="cuda")
    dy = torch.ones(5, 9, device="cuda")
    dy[0, 2] = float("inf")
    dy[4] = float("nan")
    d = msm.msm_embed_bwd(ids, dy, 4)
    assert torch.isfinite(d).all(1).tolist() == [True, True, True, False]


@pytest.mark.parametrize("T", [900, 9000])
def test_repeated_shapes_and_streams(T):
    import selective_state_space_msm_amd as msm
    gen = torch.Generator().manual_seed(T)
    ids = make("zipf", T, 1000, gen).cuda().view(3, T // 3)
    dy = torch.randn(3, T // 3, 70, generator=gen).cuda().bfloat16()
    a = msm.msm_embed_bwd(ids, dy, 1000, 0.5)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ws = torch.empty(msm.msm_embed_bwd_workspace_bytes(T, 1000, 70), dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    b = msm.msm_embed_bwd(ids, dy, 1000, 0.5, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    y = msm.msm_embed_fwd(ids, a)
    y2 = msm.msm_embed_fwd(ids, a, stream=s, io=torch.float32)
    torch.cuda.synchronize()
    assert y.shape == (3, T // 3, 70) and y.dtype is torch.bfloat16 and torch.equal(y.float(), y2)
