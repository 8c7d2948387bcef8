"""The fused norms around a block on the GPU against float64: forward, backward."""
import pytest
import torch

import lm_ref
from gpu_util import log

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# fp32: a few roundings of 2^-24 an element, the statistics' sums some more
F32 = 2e-6


def close(got, ref, what, tol):
    got = got.detach().double().cpu().reshape(ref.shape)
    assert torch.isfinite(got).all(), what
    err, norm = float((got - ref).norm()), float(ref.norm())
    log("  %s: %.2g of %.2g" % (what, err / max(norm, 1e-300), tol))
    assert err <= tol * norm + 1e-30, (what, err, norm)


def device(t, offset):
    if t is None:
        return None
    buf = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
    v = buf[offset:].view(t.shape)
    v.copy_(t)
    return v


def inputs(io, rows, D, block, gate, weights, gen):
    rnd = lambda *s: torch.randn(*s, generator=gen)
    a = dict(r=rnd(rows, D).to(DT[io]), dy=rnd(rows, D).to(DT[io]), dr=rnd(rows, D).to(DT[io]), o=None, z=None, w=None, pw=None)
    if block:
        a["o"] = (0.7 * rnd(rows, D)).to(DT[io])
    if gate:
        a["z"] = rnd(rows, D).to(DT[io])
    if weights:
        a["w"] = 1 + 0.2 * rnd(D)
        a["pw"] = 1 + 0.2 * rnd(D) if block else None
    return a


def check(io, rows, D, block=True, gate=True, weights=True, residual=True, offset=0, scale=0.6, in_place=False, eps=1e-5):
    import selective_state_space_msm_amd as msm
    gen = torch.Generator().manual_seed(rows * 7 + D)
    a = inputs(io, rows, D, block, gate, weights, gen)
    log("rows=%d D=%d %s" % (rows, D, io))
    wide = lambda t: None if t is None else t.double()
    g = {n: device(t, offset) for n, t in a.items()}
    out = 2.0 ** -8 if io == "bf16" else F32  # its rounding
    s = float(torch.tensor(scale))
    kept = g["r"].clone()
    r_out, y, rstd, q = msm.msm_block_norm_fwd(g["r"], g["w"], g["o"], g["pw"], g["z"], scale, eps=eps, return_stats=True,
                                               r_out=g["r"] if in_place else None)
    assert in_place or torch.equal(g["r"], kept)
    assert (r_out is g["r"]) == (in_place or not block)
    held = r_out.double().cpu()
    rr, ry, rrstd, rq = lm_ref.block_norm_fwd(wide(a["r"]), wide(a["w"]), wide(a["o"]), wide(a["pw"]), wide(a["z"]), s, eps, held)
    close(r_out, rr, "r_out", out)
    close(y, ry, "y", out + F32)
    close(rstd, rrstd, "rstd", F32)
    if block:
        close(q, rq, "post_rstd", F32)
        rq = rq.float()
    else:
        assert q is None
    rrstd = rrstd.float()
    d = msm.msm_block_norm_bwd(r_out, g["dy"], device(rrstd, offset), g["w"], g["o"], device(rq, offset), g["pw"], g["z"], scale,
                               dr_out=g["dr"] if residual else None)
    want = lm_ref.block_norm_bwd(held, wide(a["dy"]), wide(rrstd), wide(a["w"]), wide(a["o"]), wide(rq), wide(a["pw"]),
                                 wide(a["z"]), s, wide(a["dr"]) if residual else None)
    for n in ("dr", "do", "dz"):
        if want[n] is None:
            assert d[n] is None
        elif D > 1 or n == "dr":
            # one column: the norm's own gradient is a difference of equal terms, and only eps is left of it
            close(d[n], want[n], n, 4 * F32 + (2.0 ** -8 if io == "bf16" else 0) if D > 1 else 1e-2)
    for n, given in (("dweight", weights), ("dpost_weight", weights and block)):
        if given:
            close(d[n], want[n], n, 4 * F32)
        else:
            assert d[n] is None


SIZES = [(1, 16), (3, 17), (1, 1), (70, 24), (1000, 32), (129, 100), (5, 256), (33, 257), (300, 512), (64, 1001), (40, 2048),
         (7, 4097), (21, 4096), (9, 8192), (5, 8200), (4, 16384), (3, 20000), (2, 40001), (3001, 40)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", SIZES)
def test_sizes(io, rows, D):
    check(io, rows, D)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [128, 129, 256, 257, 512, 513, 768, 1024, 1025, 2048, 2049, 4095, 4096, 4097, 6001, 8192, 8193, 16384, 16385])
@pytest.mark.parametrize("rows", [1, 300])
def test_widths_where_the_shape_changes(io, rows, D):
    check(io, rows, D)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [48, 770, 4096, 5003, 17000])
@pytest.mark.parametrize("block,gate,weights,residual", [(False, False, True, True), (False, False, False, False),
                                                         (True, False, True, False), (True, True, False, True)])
def test_optional_inputs(io, D, block, gate, weights, residual):
    check(io, 30, D, block, gate, weights, residual)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [512, 515, 18001])
def test_unaligned(io, D):
    check(io, 20, D, offset=1)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 1001, 9000, 17001])
def test_in_place(io, D):
    check(io, 50, D, in_place=True)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [48, 300, 2000, 6000, 17000])
def test_nan_row_stays_in_its_row(io, D):
    import selective_state_space_msm_amd as msm
    gen = torch.Generator().manual_seed(D)
    a = {n: None if t is None else t.cuda() for n, t in inputs(io, 9, D, True, True, True, gen).items()}
    a["o"][3, 5] = float("nan")
    a["z"][5, 7] = float("inf")
    a["r"][7, 0] = -float("inf")
    r, y, rstd, q = msm.msm_block_norm_fwd(a["r"], a["w"], a["o"], a["pw"], a["z"], return_stats=True)
    bad = [False, False, False, True, False, True, False, True, False]
    assert (~torch.isfinite(y).all(1)).tolist() == bad
    d = msm.msm_block_norm_bwd(r, a["dy"], rstd, a["w"], a["o"], q, a["pw"], a["z"], dr_out=a["dr"])
    assert (~torch.isfinite(d["dr"]).all(1)).tolist() == bad


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_zero_rows_and_far_gates(io):
    """A row of zeros stays finite (eps), and gates of plus and minus 1e4 pass or close."""
    import selective_state_space_msm_amd as msm
    D = 256
    o, r = torch.randn(2, D, device="cuda").to(DT[io]), torch.zeros(2, D, device="cuda").to(DT[io])
    z = torch.full((2, D), -1e4, device="cuda").to(DT[io])
    r2, y, rstd, q = msm.msm_block_norm_fwd(r, None, o, None, z, eps=1e-4, return_stats=True)
    assert bool((r2 == 0).all()) and bool((y == 0).all())
    assert torch.allclose(rstd, torch.full_like(rstd, 100.0), rtol=1e-6)
    d = msm.msm_block_norm_bwd(r2, o, rstd, None, o, q, None, z)
    assert bool((d["do"] == 0).all()) and bool((d["dz"] == 0).all()) and bool(torch.isfinite(d["dr"]).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [96, 3001, 18000])
def test_repeated_and_on_another_stream(io, D):
    import selective_state_space_msm_amd as msm
    gen = torch.Generator().manual_seed(D)
    a = {n: t.cuda() for n, t in inputs(io, 300, D, True, True, True, gen).items()}
    r, y, rstd, q = msm.msm_block_norm_fwd(a["r"], a["w"], a["o"], a["pw"], a["z"], 0.3, return_stats=True)
    args = (r, a["dy"], rstd, a["w"], a["o"], q, a["pw"], a["z"], 0.3)
    d = msm.msm_block_norm_bwd(*args, dr_out=a["dr"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    r2, y2 = msm.msm_block_norm_fwd(a["r"], a["w"], a["o"], a["pw"], a["z"], 0.3, stream=s)
    d2 = msm.msm_block_norm_bwd(*args, dr_out=a["dr"], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(r, r2) and torch.equal(y, y2)
    for n in d:
        assert torch.equal(d[n], d2[n]), n


def test_column_gradients_do_not_drift():
    """40000 equal rows: a rounding of the sums' join and of each row's factors, not of 40000 additions."""
    import selective_state_space_msm_amd as msm
    rows, D = 40000, 64
    r = torch.full((rows, D), 1.1, device="cuda")
    dy = torch.full((rows, D), 0.7, device="cuda")
    rstd = torch.full((rows,), 1.3, device="cuda")
    d = msm.msm_block_norm_bwd(r, dy, rstd, torch.ones(D, device="cuda"))
    want = rows * (dy[0].double() * (r[0].double() * rstd[0].double()))
    # a thread sums at most 40000 / (512 * 8) = 10 rows; 3 roundings of a term, 10 + 4 of sums
    assert bool(((d["dweight"].double() - want).abs() <= 20 * 2.0 ** -24 * want).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1023, 1024, 1025, 2048, 2049, 4096, 4097, 8192, 8193])
def test_widths_at_which_rows_change_their_shape(io, D):
    check(io, 3, D)


@pytest.mark.parametrize("io,rows,D", [("f32", 1 << 22, 64), ("bf16", 1 << 22, 64), ("f32", 1 << 19, 520), ("bf16", 1 << 20, 1100)])
def test_column_gradients_of_many_rows_do_not_drift(io, rows, D):
    """Equal rows: a thread adds up at most 64 of them in one fp32 sum, and at most 32 such sums."""
    import selective_state_space_msm_amd as msm
    r = torch.full((rows, D), 1.1, device="cuda").to(DT[io])
    dy = torch.full((rows, D), 0.7, device="cuda").to(DT[io])
    rstd = torch.full((rows,), 1.3, device="cuda")
    d = msm.msm_block_norm_bwd(r, dy, rstd, torch.ones(D, device="cuda"))
    want = rows * (dy[0].double() * (r[0].double() * rstd[0].double()))
    # 3 roundings of a term, 64 and 32 of a thread's sums, two exchanges and four wavefronts, the result's
    assert bool(((d["dweight"].double() - want).abs() <= (3 + 64 + 32 + 6 + 1) * 2.0 ** -24 * want).all())
