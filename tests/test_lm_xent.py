"""The linear cross entropy on the GPU against float64: forward, backward."""
import pytest
import torch

import lm_ref
from gpu_util import log

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def device(t, offset=0):
    if t is None:
        return None
    buf = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
    v = buf[offset:].view(t.shape)
    v.copy_(t)
    return v


def inputs(io, T, V, D, ignored, gen, spread=2.0):
    rnd = lambda *s: torch.randn(*s, generator=gen)
    x, w = rnd(T, D).to(DT[io]), (spread * D ** -0.5 * rnd(V, D)).to(DT[io])
    t = torch.randint(V, (T,), generator=gen)
    off = torch.rand(T, generator=gen)
    t[off < ignored] = -100
    t[off < ignored / 3] = V
    return x, w, t


def ulp(n):
    return n * 2.0 ** -24


def inside(got, want, tol, what):
    got = got.detach().double().to(want.device).reshape(want.shape)
    assert torch.isfinite(got).all(), what
    err = (got - want).abs()
    log("  %s: %.2g of its bound" % (what, float((err / (tol + 1e-300)).max())))
    assert bool((err <= tol).all()), (what, float(err.max()), float((err / (tol + 1e-300)).max()))


def check(io, T, V, D, ignored=0.2, scale=0.9, penalty=True, offset=0, spread=2.0, lead=None, weight_grad=True, on="cpu"):
    import selective_state_space_msm_amd as msm
    gen = torch.Generator().manual_seed(T * 7 + V * 3 + D)
    x, w, t = inputs(io, T, V, D, ignored, gen, spread)
    log("T=%d V=%d D=%d %s" % (T, V, D, io))
    gx, gw, gt = device(x, offset), device(w, offset), t.cuda()
    if lead:
        gx, gt = gx.view(*lead, D), gt.view(lead)
    loss, lse = msm.msm_linear_cross_entropy_fwd(gx, gw, gt, scale, return_lse=True)
    assert loss.shape == gt.shape == lse.shape
    s = float(torch.tensor(scale))
    xd, wd, t = x.double().to(on), w.double().to(on), t.to(on)
    rloss, rlse, logits = lm_ref.xent_fwd(xd, wd, t, s)
    # a logit: a sum of D products, each rounding at most 2^-24 of the sum of their sizes; fp32
    # products leave out less than 2^-20 of a term and are summed in six rounds; scaling rounds once
    size = abs(s) * xd.abs() @ wd.abs().t()
    dl = (ulp(D + 2) if io == "bf16" else ulp(6 * D + 2) + 2.0 ** -20) * size
    # lse moves by the largest of these; exponentials and their sum by V roundings at most, a few in
    # earnest: 2^-20 of 1 (2^-23 an exponential, its argument's rounding); the logarithm and the sum round
    dlse = dl.max(1).values + 2.0 ** -20 + ulp(4) * logits.abs().max(1).values + ulp(4) * rlse.abs()
    live = (t >= 0) & (t < V)
    dlse = torch.where(live, dlse, 0.0)
    inside(lse, rlse, dlse, "lse")
    inside(loss, rloss, 2 * dlse, "loss")
    dloss, dp = torch.randn(T, generator=gen).to(on), (0.3 * torch.randn(T, generator=gen).to(on) if penalty else None)
    gl = rlse.float()
    shape = (lambda a: a) if not lead else (lambda a: a.view(lead))
    d = msm.msm_linear_cross_entropy_bwd(gx, gw, gt, shape(gl.cuda()), shape(dloss.cuda()), scale,
                                         dlse=None if dp is None else shape(dp.cuda()), weight_grad=weight_grad)
    g, p = lm_ref.xent_g(logits, t, gl.double(), dloss.double(), None if dp is None else dp.double(), s)
    # p = exp(l - lse): the logit's error, the difference's and the exponent's rounding, the exponential
    # (2^-22 together with both factors); then g's own rounding where it is held in bf16
    arg = (logits - gl.double()[:, None]).abs()
    dg = p.abs() * (dl + ulp(4) * (logits.abs() + arg) + 2.0 ** -21) + ulp(4) * g.abs()
    dg = dg + (2.0 ** -8 * (g.abs() + dg) if io == "bf16" else 2.0 ** -20 * g.abs())
    # what is below the smallest normal number, 2^-126, may count as zero: an exponential, g's lower parts,
    # and a product
    dg = dg + 3 * 2.0 ** -126
    tiny = 6 * (T + V) * 2.0 ** -126
    half = 2.0 ** -8 if io == "bf16" else 2.0 ** -24
    rounds = 1 if io == "bf16" else 6
    dx = g @ wd
    ga = g.abs() + dg
    tol = tiny + dg @ wd.abs() + ulp(rounds * V + 4) * (ga @ wd.abs()) + (0 if io == "bf16" else 2.0 ** -20) * (ga @ wd.abs())
    inside(d["dx"], dx, tol + half * (dx.abs() + tol), "dx")
    assert bool((d["dx"].reshape(T, D)[~live.cuda()] == 0).all())
    if not weight_grad:
        assert d["dweight"] is None
        return
    xa = xd.abs()
    dw = g.t() @ xd
    tol = tiny + dg.t() @ xa + (ulp(rounds * T + 4) + (0 if io == "bf16" else 2.0 ** -20)) * (ga.t() @ xa)
    inside(d["dweight"], dw, tol + half * (dw.abs() + tol), "dweight")


SIZES = [(1, 1, 1), (1, 2, 8), (3, 5, 7), (17, 100, 16), (2, 257, 33), (64, 64, 64), (65, 129, 72), (130, 300, 63),
         (128, 128, 128), (200, 1000, 65), (300, 513, 200), (1, 3001, 96), (16, 5000, 136), (257, 257, 264)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_sizes(io, T, V, D):
    check(io, T, V, D)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,D", [(513, 32801, 72), (1030, 13000, 264)])
def test_many_tiles(io, T, V, D):
    check(io, T, V, D)


@pytest.mark.parametrize("io,T,V,D", [("bf16", 2048, 8200, 584), ("bf16", 2056, 1030, 8192), ("bf16", 1030, 2056, 8200),
                                      ("bf16", 900, 3001, 1032), ("f32", 1800, 1700, 100), ("f32", 300, 6000, 1030)])
def test_tiles_of_every_size(io, T, V, D):
    """Logits, dx and dweight in tiles of 256 each once, and in tiles of 128 and 64; the float64 products on the GPU."""
    check(io, T, V, D, on="cuda")


@pytest.mark.parametrize("T", [1, 2, 5, 16, 17, 31, 32, 33, 48, 64, 65])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_few_rows(io, T):
    check(io, T, 4099, 192, ignored=0.1)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 61])
def test_unaligned(io, D):
    check(io, 70, 700, D, offset=1)
    check(io, 5, 700, D, offset=1)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_leading_dimensions_and_options(io):
    check(io, 60, 90, 40, lead=(3, 4, 5), penalty=False)
    check(io, 60, 90, 40, weight_grad=False)
    check(io, 60, 90, 40, ignored=0.0, scale=-1.3)
    check(io, 60, 90, 40, scale=0.0)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_far_logits(io):
    """Logits of some hundred: exponentials of all but the largest vanish."""
    check(io, 40, 600, 64, spread=60.0)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [6, 300])
def test_rows_left_out_hold_anything(io, T):
    import selective_state_space_msm_amd as msm
    gen = torch.Generator().manual_seed(T)
    x, w, t = inputs(io, T, 500, 72, 0.4, gen)
    t[1], t[2] = -1, 500
    live = ((t >= 0) & (t < 500)).cuda()
    x, w, t = x.cuda(), w.cuda(), t.cuda()
    dl = torch.randn(T, generator=gen).cuda()
    loss, lse = msm.msm_linear_cross_entropy_fwd(x, w, t, return_lse=True)
    d = msm.msm_linear_cross_entropy_bwd(x, w, t, lse, dl, dlse=dl)
    nan = float("nan")
    x2, dl2, lse2 = x.clone(), dl.clone(), lse.clone()
    x2[~live] = nan
    dl2[~live] = nan
    lse2[~live] = nan
    loss2, l2 = msm.msm_linear_cross_entropy_fwd(x2, w, t, return_lse=True)
    d2 = msm.msm_linear_cross_entropy_bwd(x2, w, t, lse2, dl2, dlse=dl2)
    assert torch.equal(loss, loss2) and torch.equal(lse, l2)
    assert torch.equal(d["dx"], d2["dx"]) and torch.equal(d["dweight"], d2["dweight"])
    assert bool((loss[~live] == 0).all()) and bool((lse[~live] == 0).all()) and bool((d2["dx"][~live] == 0).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_no_row_with_a_target(io):
    import selective_state_space_msm_amd as msm
    x, w = torch.full((150, 64), float("nan"), device="cuda").to(DT[io]), torch.randn(300, 64, device="cuda").to(DT[io])
    t = torch.full((150,), -100, device="cuda")
    one = torch.ones(150, device="cuda")
    loss = msm.msm_linear_cross_entropy_fwd(x, w, t)
    d = msm.msm_linear_cross_entropy_bwd(x, w, t, one, one)
    assert bool((loss == 0).all()) and bool((d["dx"] == 0).all()) and bool((d["dweight"] == 0).all())


@pytest.mark.parametrize("io,T,V,D,ignored", [("bf16", 4100, 17000, 64, 0.97), ("bf16", 9000, 33000, 40, 0.9995),
                                              ("bf16", 2300, 4200, 1032, 0.8), ("f32", 2500, 9000, 33, 0.9)])
def test_most_rows_left_out(io, T, V, D, ignored):
    """Far fewer tiles of rows than the launch is made for."""
    check(io, T, V, D, ignored=ignored, on="cuda")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,D", [(600, 1000, 64), (520, 8000, 136), (2100, 2048, 264), (513, 64, 1)])
def test_no_row_of_many_with_a_target(io, T, V, D):
    """More rows than stay in their places: none are gathered, the products have no tiles of rows."""
    import selective_state_space_msm_amd as msm
    x, w = torch.full((T, D), float("nan"), device="cuda").to(DT[io]), torch.randn(V, D, device="cuda").to(DT[io])
    t = torch.full((T,), V, device="cuda")
    one = torch.ones(T, device="cuda")
    loss, lse = msm.msm_linear_cross_entropy_fwd(x, w, t, return_lse=True)
    d = msm.msm_linear_cross_entropy_bwd(x, w, t, one, one, dlse=one)
    assert bool((loss == 0).all()) and bool((lse == 0).all())
    assert bool((d["dx"] == 0).all()) and bool((d["dweight"] == 0).all())


@pytest.mark.parametrize("T", [4, 200])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_nan_row_stays_in_its_row(io, T):
    import selective_state_space_msm_amd as msm
    gen = torch.Generator().manual_seed(T)
    x, w, t = inputs(io, T, 400, 64, 0.0, gen)
    x[2, 5] = float("nan")
    loss, lse = msm.msm_linear_cross_entropy_fwd(x.cuda(), w.cuda(), t.cuda(), return_lse=True)
    bad = torch.zeros(T, dtype=torch.bool)
    bad[2] = True
    assert torch.equal(torch.isnan(loss).cpu(), bad) and torch.equal(torch.isnan(lse).cpu(), bad)
    d = msm.msm_linear_cross_entropy_bwd(x.cuda(), w.cuda(), t.cuda(), lse, torch.ones(T, device="cuda"))
    assert torch.equal(torch.isnan(d["dx"]).any(1).cpu(), bad)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [8, 500])
def test_lowest_logits(io, T):
    """A weight row whose logits are the lowest number there is, or minus infinity: a probability of 0."""
    import selective_state_space_msm_amd as msm
    x = torch.rand(T, 64, device="cuda").to(DT[io])
    w = torch.randn(300, 64, device="cuda").to(DT[io])
    t = torch.randint(299, (T,), device="cuda")
    low = torch.finfo(torch.float32).min
    # an infinite fp32 value has no parts: bf16 alone
    for value in (-1e30, low / 64, -float("inf"))[: 3 if io == "bf16" else 2]:
        v = w.clone()
        v[299] = torch.tensor(value).to(DT[io])
        loss, lse = msm.msm_linear_cross_entropy_fwd(x, v, t, return_lse=True)
        rest, rest_lse = msm.msm_linear_cross_entropy_fwd(x, w[:299].contiguous(), t, return_lse=True)
        assert torch.allclose(loss, rest, rtol=1e-5, atol=1e-5) and torch.allclose(lse, rest_lse, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("T", [8, 500, 700])
def test_left_out_rows_add_nothing_to_infinite_weights(T):
    """A weight row of minus infinity, a probability of 0 in every row: its gradient is 0, and the others' is as
    it is without that row, also where rows are left out."""
    import selective_state_space_msm_amd as msm
    x, w = (torch.rand(T, 64, device="cuda") + 0.1).bfloat16(), torch.randn(300, 64, device="cuda").bfloat16()
    w[299] = -float("inf")
    t = torch.randint(299, (T,), device="cuda")
    t[::3] = -1
    one = torch.ones(T, device="cuda")
    loss, lse = msm.msm_linear_cross_entropy_fwd(x, w, t, return_lse=True)
    d = msm.msm_linear_cross_entropy_bwd(x, w, t, lse, one, dlse=one)
    rest = msm.msm_linear_cross_entropy_bwd(x, w[:299].contiguous(), t, lse, one, dlse=one)
    assert bool((d["dweight"][299] == 0).all()) and bool((d["dx"][::3] == 0).all())
    assert torch.equal(d["dweight"][:299], rest["dweight"])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [16, 400])
def test_repeated_and_on_another_stream(io, T):
    import selective_state_space_msm_amd as msm
    gen = torch.Generator().manual_seed(T)
    x, w, t = (a.cuda() for a in inputs(io, T, 3001, 200, 0.2, gen))
    dl = torch.randn(T, generator=gen).cuda()
    loss, lse = msm.msm_linear_cross_entropy_fwd(x, w, t, return_lse=True)
    d = msm.msm_linear_cross_entropy_bwd(x, w, t, lse, dl)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    loss2 = msm.msm_linear_cross_entropy_fwd(x, w, t, stream=s)
    d2 = msm.msm_linear_cross_entropy_bwd(x, w, t, lse, dl, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(loss, loss2) and torch.equal(d["dx"], d2["dx"]) and torch.equal(d["dweight"], d2["dweight"])
    # a workspace of other calls' remains
    need = msm.msm_linear_cross_entropy_bwd_workspace_bytes(T, 3001, 200, DT[io])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    d3 = msm.msm_linear_cross_entropy_bwd(x, w, t, lse, dl, workspace=ws)
    assert torch.equal(d["dx"], d3["dx"]) and torch.equal(d["dweight"], d3["dweight"])
