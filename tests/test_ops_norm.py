"""Layer norm on the GPU against float64: forward, backward."""
import pytest
import torch

import ops_ref
from gpu_util import log

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def close(got, ref, what, tol):
    got = got.detach().double().cpu().reshape(ref.shape)
    assert torch.isfinite(got).all(), what
    err, norm = float((got - ref).norm()), float(ref.norm())
    log("  %s: %.2g of %.2g" % (what, err / max(norm, 1e-300), tol))
    assert err <= tol * norm + 1e-30, (what, err, norm)


def device(t, offset):
    buf = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
    v = buf[offset:].view(t.shape)
    v.copy_(t)
    return v


def check(io, rows, D, weight=True, bias=True, shift=0.3, offset=0, eps=1e-5):
    import selective_state_space_msm_amd as msm
    gen = torch.Generator().manual_seed(rows * 7 + D)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    x, dy = (rnd(rows, D) + shift).to(DT[io]), rnd(rows, D).to(DT[io])
    w, b = (1 + 0.2 * rnd(D)) if weight else None, rnd(D) if bias else None
    log("rows=%d D=%d %s" % (rows, D, io))
    wide = lambda t: None if t is None else t.double()
    gpu = lambda t: None if t is None else device(t, offset)
    y, mean, rstd = msm.msm_layer_norm_fwd(gpu(x), gpu(w), gpu(b), eps=eps, return_stats=True)
    ry, rmean, rrstd = ops_ref.norm_fwd(wide(x), wide(w), wide(b), eps)
    # fp32: a few roundings of 2^-24, x - mean magnified by |mean| / sigma; a sum over a row or
    # over all rows adds sqrt(n) of them at most, and cancels to its size over sqrt(n) at worst
    f32 = 2e-6 * (1 + abs(shift))
    out = f32 if io == "f32" else 2.2e-3  # bf16: its rounding, 2^-9 at most
    close(y, ry, "y", out)
    close(mean, rmean, "mean", f32 if abs(shift) >= 0.3 else 1e-5)
    close(rstd, rrstd, "rstd", f32)
    mean, rstd = rmean.float(), rrstd.float()
    d = msm.msm_layer_norm_bwd(gpu(x), gpu(dy), gpu(mean), gpu(rstd), gpu(w), bias_grad=bias)
    rdx, rdw, rdb = ops_ref.norm_bwd(wide(x), wide(w), wide(dy), wide(mean), wide(rstd))
    close(d["dx"], rdx, "dx", 4 * f32 if io == "f32" else 2.2e-3)
    if weight:
        close(d["dweight"], rdw, "dweight", 4 * f32)
    else:
        assert d["dweight"] is None
    if bias:
        close(d["dbias"], rdb, "dbias", 4 * f32)
    else:
        assert d["dbias"] is None


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", [(1, 16), (3, 17), (70, 24), (1000, 32), (129, 100), (5, 256), (33, 257),
                                    (300, 512), (64, 1000), (40, 2048), (7, 4097), (21, 4096), (9, 8192),
                                    (4, 16384), (3, 20000), (2, 40000), (70, 5001), (3000, 40)])
def test_sizes(io, rows, D):
    check(io, rows, D)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_optional_parameters(weight, bias):
    check("bf16", 50, 768, weight, bias)
    check("f32", 50, 768, weight, bias)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_unaligned(io):
    check(io, 20, 512, offset=1)


def test_large_mean():
    check("f32", 30, 1024, shift=30.0)


def test_constant_rows_and_one_column():
    """No variance: rstd = 1 / sqrt(eps), y = bias and dx = 0 exactly."""
    import selective_state_space_msm_amd as msm
    for D in (1, 64, 2048):
        x = torch.full((5, D), 1.5, device="cuda")
        b = torch.randn(D, device="cuda")
        y, mean, rstd = msm.msm_layer_norm_fwd(x, None, b, eps=1e-4, return_stats=True)
        assert torch.equal(y, b.expand(5, D)) and torch.equal(mean, x[:, 0])
        assert torch.allclose(rstd, torch.full_like(rstd, 100.0), rtol=1e-6)
    d = msm.msm_layer_norm_bwd(x[:, :1].contiguous(), torch.ones(5, 1, device="cuda"), mean, rstd)
    assert bool((d["dx"] == 0).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_nan_row_stays_in_its_row(io):
    import selective_state_space_msm_amd as msm
    x = torch.randn(8, 48, device="cuda").to(DT[io])
    x[3, 5] = float("nan")
    x[5, 7] = float("inf")
    y = msm.msm_layer_norm_fwd(x)
    bad = ~torch.isfinite(y).all(1)
    assert bad.tolist() == [False, False, False, True, False, True, False, False]


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_repeated_and_on_another_stream(io):
    import selective_state_space_msm_amd as msm
    x, dy = (torch.randn(500, 96, device="cuda").to(DT[io]) for _ in range(2))
    w = torch.randn(96, device="cuda")
    y, mean, rstd = msm.msm_layer_norm_fwd(x, w, return_stats=True)
    a = msm.msm_layer_norm_bwd(x, dy, mean, rstd, w, bias_grad=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2 = msm.msm_layer_norm_fwd(x, w, stream=s)
    b = msm.msm_layer_norm_bwd(x, dy, mean, rstd, w, bias_grad=True, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_column_gradients_of_very_wide_rows():
    """2^28 columns: a workgroup for 16 of them would make 2^32 threads, more than a launch may have."""
    import selective_state_space_msm_amd as msm
    D = 1 << 28
    x = torch.randn(1, D, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(1, D, device="cuda", dtype=torch.bfloat16)
    mean, rstd = torch.full((1,), 0.25, device="cuda"), torch.full((1,), 1.5, device="cuda")
    nan = lambda: torch.full((D,), float("nan"), device="cuda")
    out = {"dweight": nan(), "dbias": nan()}
    d = msm.msm_layer_norm_bwd(x, dy, mean, rstd, torch.ones(D, device="cuda"), bias_grad=True, out=out)
    assert torch.equal(d["dbias"], dy[0].float())
    # one product of two roundings each
    want = dy[0].float() * ((x[0].float() - 0.25) * 1.5)
    assert bool(((d["dweight"] - want).abs() <= 2.0 ** -22 * want.abs()).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_long_rows(io):
    """Rows past the registers: a thread's own sum has thousands of terms.  For equal terms the
    roundings of an fp32 sum all go one way; mean, variance and column sums must not drift with them."""
    import selective_state_space_msm_amd as msm
    D = (1 << 22) + 3
    x = torch.full((2, D), 1.1, device="cuda").to(DT[io])
    b = torch.randn(D, device="cuda")
    y, mean, rstd = msm.msm_layer_norm_fwd(x, None, b, eps=1e-4, return_stats=True)
    assert torch.equal(mean, x[:, 0].float())
    assert torch.equal(y, b.to(DT[io]).expand(2, D))
    assert torch.allclose(rstd, torch.full_like(rstd, 100.0), rtol=1e-6)
    # u = 0.7 everywhere and xh = 0.5: dx = rstd (u - u - xh mean(u xh)) = -0.175 rstd
    dy = torch.full((2, D), 0.7, device="cuda").to(DT[io])
    mean, rstd = x[:, 0].float() - 0.5, torch.ones(2, device="cuda")
    dx = msm.msm_layer_norm_bwd(x, dy, mean, rstd)["dx"]
    want = -0.25 * dy.double()
    tol = 1e-6 if io == "f32" else 2.0 ** -8
    assert bool(((dx.double() - want).abs() <= tol * want.abs()).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_column_gradients_over_many_wide_rows(io):
    import selective_state_space_msm_amd as msm
    rows, D = 40000, 4097 if io == "bf16" else 16385
    x = torch.full((rows, D), 1.1, device="cuda").to(DT[io])
    dy = torch.full((rows, D), 0.7, device="cuda").to(DT[io])
    mean, rstd = torch.full((rows,), 0.4, device="cuda"), torch.full((rows,), 1.3, device="cuda")
    d = msm.msm_layer_norm_bwd(x, dy, mean, rstd, torch.ones(D, device="cuda"), bias_grad=True)
    # a rounding of the sum and two of xh
    db = rows * dy[0].double()
    dw = db * ((x[0].float() - 0.4) * 1.3).double()
    assert bool(((d["dbias"].double() - db).abs() <= 2.0 ** -22 * db).all())
    assert bool(((d["dweight"].double() - dw).abs() <= 2.0 ** -22 * dw).all())
