"""Gated delta rule on the GPU against the float64 recurrence: forward, backward, one token."""
import pytest
import torch

import ops_ref
from gpu_util import log

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}

# Bounds on the 2-norm of the error over the 2-norm of the result.
#   fp32 results: sums of at most 256 + 64 terms rounded to 2^-24, chained over the solve, the
#   state and the readout, whose factors here are at most about 8 (unit keys, beta < 1):
#   6e-8 * sqrt(320) * 8 = 9e-6.
#   bf16 results: the rounding of the result itself, at most 2^-9 of each element, 2e-3, and the
#   16-bit parts it is made of, 2^-15 of the larger terms they cancel from: 2.5e-3 in all.
TOL = {torch.float32: 1e-5, torch.bfloat16: 2.5e-3}


def make(io, lens, Hk, H, K, V, seed=0, packed=False, g_scale=1.0):
    gen = torch.Generator().manual_seed(1000 + seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    T = sum(lens)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)
    d = dict(q=unit(rnd(T, Hk, K)).to(DT[io]), k=unit(rnd(T, Hk, K)).to(DT[io]),
             v=rnd(T, H, V).to(DT[io]), g=-g_scale * torch.rand(T, H, generator=gen) ** 2,
             beta=torch.sigmoid(rnd(T, H)), S0=0.3 * rnd(len(lens), H, K, V),
             do=rnd(T, H, V).to(DT[io]), dlast=rnd(len(lens), H, K, V), lens=lens, packed=packed)
    return d


def to_gpu(d, offset=0):
    """Device copies; `offset` elements past an aligned address."""
    out = {}
    n = len(d["lens"])
    for name, t in d.items():
        if not torch.is_tensor(t):
            continue
        if not d["packed"] and name in ("q", "k", "v", "g", "beta", "do"):
            t = t.reshape((n, d["lens"][0]) + t.shape[1:])
        buf = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
        out[name] = buf[offset:].view(t.shape)
        out[name].copy_(t)
    if d["packed"]:
        ends = [0]
        for l in d["lens"]:
            ends.append(ends[-1] + l)
        out["off"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    else:
        out["off"] = None
    return out


def want(d, scale, bwd, S0=True, dlast=True):
    """References of all sequences, packed one after the other."""
    w = {n: t.double() for n, t in d.items() if torch.is_tensor(t)}
    parts, at = [], 0
    for b, l in enumerate(d["lens"]):
        e = slice(at, at + l)
        at += l
        s0 = w["S0"][b] if S0 else None
        seq = [w[n][e] for n in ("q", "k", "v", "g", "beta")]
        if bwd:
            parts.append(ops_ref.delta_bwd(*seq, scale, w["do"][e], s0, w["dlast"][b] if dlast else None))
        else:
            o, S, _ = ops_ref.delta_fwd(*seq, scale, s0)
            parts.append(dict(o=o, S=S))
    stack = ("S", "dS0")
    return {n: (torch.stack if n in stack else torch.cat)([p[n] for p in parts]) for n in parts[0]}


def close(got, ref, what, tol=None):
    tol = TOL[got.dtype] if tol is None else tol
    got = got.detach().double().cpu().reshape(ref.shape)
    assert torch.isfinite(got).all(), what
    err, norm = float((got - ref).norm()), float(ref.norm())
    log("  %s: %.2g of %.2g" % (what, err / max(norm, 1e-300), tol))
    assert err <= tol * norm + 1e-30, (what, err, norm)


def run_fwd(d, offset=0, **kw):
    import selective_state_space_msm_amd as msm
    t = to_gpu(d, offset)
    o, S = msm.msm_delta_rule_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], S0=t["S0"],
                                  seq_offsets=t["off"], return_last_state=True, **kw)
    torch.cuda.synchronize()
    return o, S


def run_bwd(d, offset=0, **kw):
    import selective_state_space_msm_amd as msm
    t = to_gpu(d, offset)
    r = msm.msm_delta_rule_bwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["do"], S0=t["S0"],
                               dlast_S=t["dlast"], seq_offsets=t["off"], state_grads=True, **kw)
    torch.cuda.synchronize()
    return r


def check(d, offset=0, tol=None):
    log("lens=%s q=%s v=%s %s" % (d["lens"], tuple(d["q"].shape), tuple(d["v"].shape), d["v"].dtype))
    scale = d["q"].shape[-1] ** -0.5
    o, S = run_fwd(d, offset)
    ref = want(d, scale, False)
    close(o, ref["o"], "o", tol)
    close(S, ref["S"], "last_S", tol)
    got = run_bwd(d, offset)
    ref = want(d, scale, True)
    for n in ref:
        close(got[n], ref[n], n, tol)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 15, 31, 32, 33, 63, 64, 65, 127, 129, 200])
def test_lengths(io, L):
    check(make(io, [L, L], 2, 2, 32, 32, seed=L))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", [(1, 1), (7, 5), (16, 40), (33, 17), (64, 64), (72, 130), (128, 128),
                                 (130, 24), (200, 63), (256, 256)])
def test_head_sizes(io, K, V):
    check(make(io, [70, 70], 1, 2, K, V, seed=K + V))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Hk,H", [(1, 1), (1, 4), (3, 6), (2, 10)])
def test_shared_heads(io, Hk, H):
    check(make(io, [67], Hk, H, 48, 24, seed=H))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[5], [1, 1, 1], [0, 1, 64, 65, 0, 130, 0], [63, 128, 2], [0, 7]])
def test_packed(io, lens):
    check(make(io, lens, 2, 4, 64, 48, seed=sum(lens), packed=True))


def test_packed_empty_sequence_keeps_its_state():
    d = make("bf16", [0, 40, 0], 1, 2, 32, 32, packed=True)
    o, S = run_fwd(d)
    assert torch.equal(S[0].cpu(), d["S0"][0]) and torch.equal(S[2].cpu(), d["S0"][2])
    r = run_bwd(d)
    assert torch.equal(r["dS0"][0].cpu(), d["dlast"][0]) and torch.equal(r["dS0"][2].cpu(), d["dlast"][2])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_unaligned_arrays(io):
    check(make(io, [70, 70], 1, 2, 64, 64, seed=5), offset=1)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_no_states(io):
    """No initial state, no adjoint of the last one, and the state outputs left out."""
    import selective_state_space_msm_amd as msm
    d = make(io, [90, 90], 2, 2, 40, 40, seed=6)
    t = to_gpu(d)
    o = msm.msm_delta_rule_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], 0.3)
    close(o, want(d, 0.3, False, S0=False)["o"], "o")
    r = msm.msm_delta_rule_bwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["do"], 0.3)
    assert "dS0" not in r
    ref = want(d, 0.3, True, S0=False, dlast=False)
    for n in r:
        close(r[n], ref[n], n)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["no_decay", "strong_decay", "beta_zero", "same_keys", "zero_keys"])
def test_extremes(io, kind):
    d = make(io, [150], 1, 2, 32, 32, seed=8)
    tol = None
    if kind == "no_decay":
        d["g"].zero_()
    elif kind == "strong_decay":
        d["g"] = -60 * torch.rand(150, 2)
    elif kind == "beta_zero":
        d["beta"][20:90] = 0
    elif kind == "zero_keys":
        d["k"][10:100] = 0
    elif kind == "same_keys":
        # one key throughout and full writes: the system is (all ones below the diagonal), whose
        # condition number is about the chunk length, 64: the bound grows by 8 for the sum of
        # that many alike terms
        d["k"][:] = d["k"][:1]
        d["beta"].fill_(1.0)
        d["g"].zero_()
        tol = {torch.float32: 8e-5, torch.bfloat16: 2.5e-3}[DT[io]]
    if kind == "same_keys":
        o, S = run_fwd(d)
        ref = want(d, 32 ** -0.5, False)
        close(o, ref["o"], "o", tol)
        close(S, ref["S"], "last_S", 8e-5)
    else:
        check(d)


@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.float32).min, -1e5])
def test_reset(low):
    """A decay of minus infinity, or the lowest float, forgets everything before its token; the
    decays after it keep their values."""
    d = make("f32", [100], 1, 2, 32, 32, seed=9)
    d["g"][37] = low
    d["g"][70] = low
    o, S = run_fwd(d)
    d2 = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in d.items()}
    d2["g"][37] = d2["g"][70] = -2e3  # exp is 0 in float64 too
    ref = want(d2, 32 ** -0.5, False)
    close(o, ref["o"], "o")
    close(S, ref["S"], "last_S")
    got, ref = run_bwd(d), want(d2, 32 ** -0.5, True)
    for n in ref:
        close(got[n], ref[n], n)


def test_rows_outside_the_sequences_are_not_read():
    """Packed rows past the last offset may hold anything."""
    import selective_state_space_msm_amd as msm
    d = make("bf16", [70], 1, 2, 32, 32, seed=10, packed=True)
    t = to_gpu(d)
    pad = lambda x: torch.cat([x, torch.full((30,) + x.shape[1:], float("nan"), dtype=x.dtype, device="cuda")])
    o, S = msm.msm_delta_rule_fwd(pad(t["q"]), pad(t["k"]), pad(t["v"]), pad(t["g"]), pad(t["beta"]),
                                  S0=t["S0"], seq_offsets=t["off"], return_last_state=True)
    ref = want(d, 32 ** -0.5, False)
    close(o[:70], ref["o"], "o")
    close(S, ref["S"], "last_S")


@pytest.mark.parametrize("ends", [[0, 500, 3], [-7, 40, 2 ** 31 - 1], [60, 20, 70]])
def test_wrong_offsets_stay_inside_the_arrays(ends):
    """Offsets out of range or out of order are clamped: the call ends and touches nothing else."""
    import selective_state_space_msm_amd as msm
    d = make("bf16", [35, 35], 1, 2, 32, 32, seed=11, packed=True)
    t = to_gpu(d)
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    guard = torch.full((70 + 64, 2, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    msm.msm_delta_rule_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], seq_offsets=off, o=guard[:70])
    torch.cuda.synchronize()
    assert bool((guard[70:] == 7.0).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_repeated_and_on_another_stream(io):
    """Same bits on every run, whatever the workspace held, and on a side stream."""
    import selective_state_space_msm_amd as msm
    d = make(io, [130, 130], 2, 4, 64, 80, seed=12)
    t = to_gpu(d)
    args = (t["q"], t["k"], t["v"], t["g"], t["beta"])
    n = msm.msm_delta_rule_bwd_workspace_bytes(2, 130, 2, 4, 64, 80, io)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    a = msm.msm_delta_rule_bwd(*args, t["do"], S0=t["S0"], dlast_S=t["dlast"], state_grads=True,
                               workspace=ws)
    o = msm.msm_delta_rule_fwd(*args, S0=t["S0"], workspace=ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = msm.msm_delta_rule_bwd(*args, t["do"], S0=t["S0"], dlast_S=t["dlast"], state_grads=True, stream=s)
    o2 = msm.msm_delta_rule_fwd(*args, S0=t["S0"], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(o, o2)
    for name in a:
        assert torch.equal(a[name], b[name]), name


def test_split_sequence_continues():
    """Two calls, the second from the first one's state, give one call's result."""
    import selective_state_space_msm_amd as msm
    d = make("f32", [180], 1, 2, 64, 32, seed=13)
    t = to_gpu(d)
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    o, S = msm.msm_delta_rule_fwd(*args, return_last_state=True)
    o1, S1 = msm.msm_delta_rule_fwd(*(x[:, :77].contiguous() for x in args), return_last_state=True)
    o2, S2 = msm.msm_delta_rule_fwd(*(x[:, 77:].contiguous() for x in args), S0=S1, return_last_state=True)
    close(torch.cat([o1, o2], 1), o.double().cpu(), "o")
    close(S2, S.double().cpu(), "last_S")


def test_directional_derivative():
    """The backward against differences of the forward.  In fp32 the difference of two losses of
    size |loss| carries 2^-24 sqrt(n) |terms| of noise; with a step of 1e-2 the truncation is
    ~1e-4 relative and the noise below that."""
    import selective_state_space_msm_amd as msm
    d = make("f32", [100], 1, 2, 32, 32, seed=14)
    t = to_gpu(d)
    names = ("q", "k", "v", "g", "beta", "S0")

    def loss(x):
        o, S = msm.msm_delta_rule_fwd(*(x[n] for n in names[:5]), S0=x["S0"], return_last_state=True)
        return float((o.double() * t["do"].double()).sum() + (S.double() * t["dlast"].double()).sum())

    r = run_bwd(d)
    gen = torch.Generator().manual_seed(15)
    for n in names:
        u = torch.randn(t[n].shape, generator=gen).cuda() * (0.1 if n in ("g", "beta") else 1.0)
        h = 1e-2
        num = (loss(dict(t, **{n: t[n] + h * u})) - loss(dict(t, **{n: t[n] - h * u}))) / (2 * h)
        got = float((r["d" + n].double().reshape(u.shape) * u.double()).sum())
        size = float((r["d" + n].double().reshape(u.shape).norm() * u.double().norm()))
        log("  d%s: %.6g vs %.6g" % (n, got, num))
        assert abs(got - num) <= 2e-3 * max(abs(num), 0.05 * size), n


# ---- one token -------------------------------------------------------------------------------

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Bt,Hk,H,K,V,offset", [(1, 1, 1, 1, 1, 0), (3, 2, 4, 16, 20, 0), (2, 1, 3, 33, 7, 0),
                                                (5, 2, 2, 64, 64, 0), (2, 2, 4, 128, 128, 0),
                                                (1, 1, 2, 200, 130, 0), (2, 1, 1, 256, 256, 0),
                                                (2, 2, 4, 128, 128, 1), (130, 2, 4, 64, 128, 0),
                                                (300, 1, 2, 72, 65, 0), (140, 2, 4, 256, 72, 0)])
def test_step(io, Bt, Hk, H, K, V, offset):
    import selective_state_space_msm_amd as msm
    d = make(io, [1] * Bt, Hk, H, K, V, seed=Bt + K + V, packed=True)
    t = to_gpu(d, offset)
    ref = want(d, K ** -0.5, False)
    o = msm.msm_delta_rule_step(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"])
    torch.cuda.synchronize()
    log("step %s" % ((Bt, Hk, H, K, V, offset),))
    close(o, ref["o"], "o")
    close(t["S0"], ref["S"], "S")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Bt,H,V,offset", [((1 << 24) + 3, 1, 1, 0), ((1 << 23) + 1, 2, 2, 0),
                                           (1, 1, 1 << 20, 0), (1, 1, 1 << 20, 1)])
def test_step_of_many_sequences_or_columns(io, Bt, H, V, offset):
    """More states than a launch of one workgroup each may have, and the widest state."""
    import selective_state_space_msm_amd as msm
    gen = torch.Generator("cuda").manual_seed(22)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    q, k, v = rnd(Bt, H, 1).to(DT[io]), rnd(Bt, H, 1).to(DT[io]), rnd(Bt, H, V).to(DT[io])
    g, beta = -rnd(Bt, H).square(), torch.sigmoid(rnd(Bt, H))
    S = torch.empty(Bt * H * V + offset, device="cuda")[offset:].view(Bt, H, 1, V).copy_(rnd(Bt, H, 1, V))
    qw, kw, vw, Sw = (t.double() for t in (q, k, v, S))
    Sw = g.double().exp()[..., None, None] * Sw
    Sw = Sw + (kw * beta.double()[..., None] * (vw - kw * Sw[..., 0, :]))[..., None, :]
    o = msm.msm_delta_rule_step(q, k, v, g, beta, S)
    torch.cuda.synchronize()
    close(o, (qw * Sw[..., 0, :]).cpu(), "o")
    close(S, Sw.cpu(), "S")


def test_prefill_then_steps():
    import selective_state_space_msm_amd as msm
    d = make("bf16", [80, 80], 2, 4, 64, 64, seed=21)
    t = to_gpu(d)
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    _, S = msm.msm_delta_rule_fwd(*(x[:, :70].contiguous() for x in args), S0=t["S0"], return_last_state=True)
    o = [msm.msm_delta_rule_step(*(x[:, i].contiguous() for x in args), S) for i in range(70, 80)]
    ref = want(d, 64 ** -0.5, False)
    close(torch.stack(o, 1), ref["o"].reshape(2, 80, 4, 64)[:, 70:], "o")
    close(S, ref["S"], "S")


# ---- sequences cut into segments ---------------------------------------------------------------

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens,packed", [([2100], False), ([1600, 1600], False), ([1700, 0, 512, 1, 1900], True)])
def test_segments(io, lens, packed):
    """Few heads and long sequences: the walk is cut and joined."""
    check(make(io, lens, 1, 2, 64, 40, seed=len(lens), packed=packed, g_scale=0.02))


def test_segments_of_wide_heads():
    check(make("bf16", [1800], 1, 1, 128, 80, seed=31, g_scale=0.01))
    check(make("f32", [900], 1, 1, 200, 33, seed=32, g_scale=0.01))  # chunks of 32


# ---- bf16 results ------------------------------------------------------------------------------

@pytest.mark.parametrize("Hk,H,K,V", [(2, 4, 64, 64), (1, 2, 128, 128), (1, 1, 256, 80)])
def test_bf16_results_are_the_rounded_ones(Hk, H, K, V):
    """bf16 I/O is rounded once, from fp32 accuracy.  A sum of 320 terms in fp32 is off by
    e = 6e-8 sqrt(320) of its size; an error e x moves a value x to the neighbouring bf16, a step of at
    most 2^-7 x away, with a probability of e x / step, so the 2-norm of the difference to the rounded
    float64 results is at most sqrt(2^-7 e) of theirs."""
    tol = (2.0 ** -7 * 6e-8 * 320 ** 0.5) ** 0.5
    d = make("bf16", [200, 130], Hk, H, K, V, seed=40 + K, packed=True, g_scale=0.1)
    got = dict(run_bwd(d), o=run_fwd(d)[0])
    ref = dict(want(d, K ** -0.5, True), **want(d, K ** -0.5, False))
    for n in ("o", "dq", "dk", "dv"):
        close(got[n], ref[n].bfloat16().double(), n, tol)


# ---- more of the builds and of the inputs ------------------------------------------------------

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens,K,V", [([1700], 24, 40), ([1650, 1600], 100, 24), ([1700], 100, 130), ([1700], 140, 40)])
def test_segments_of_every_build(io, lens, K, V):
    """Keys padded to 32, 128 and 256; ragged last chunks, one and two sequences."""
    check(make(io, lens, 1, 1, K, V, seed=50 + K, packed=len(lens) > 1, g_scale=0.02))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", [(32, 32), (128, 64)])
def test_write_strengths_up_to_two(io, K, V):
    """beta in (0, 2): 1 - beta |k|^2 stays within -1 and 1, so a state still forgets, but a write is up
    to twice as large: twice the fp32 bound."""
    d = make(io, [150, 90], 1, 2, K, V, seed=60 + K, packed=True, g_scale=0.1)
    d["beta"] = 2 * d["beta"]
    check(d, tol=None if io == "bf16" else 2 * TOL[torch.float32])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["no_decay", "strong_decay", "beta_zero"])
def test_extremes_of_wide_heads(io, kind):
    d = make(io, [150], 1, 2, 128, 96, seed=61)
    if kind == "no_decay":
        d["g"].zero_()
    elif kind == "strong_decay":
        d["g"] = -60 * torch.rand(150, 2)
    else:
        d["beta"][20:90] = 0
    check(d)


def test_backward_of_alike_keys():
    """One key throughout and full writes, as in the forward's test: the errors pass through the chunk's
    system twice, once for e and once, transposed, for dv, each time up to 8 times as large."""
    d = make("f32", [150], 1, 2, 32, 32, seed=8)
    d["k"][:] = d["k"][:1]
    d["beta"].fill_(1.0)
    d["g"].zero_()
    check(d, tol=64 * TOL[torch.float32])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_lowest_values_that_are_never_written(io):
    """A value of the type's lowest at a token with beta = 0 and no adjoint changes nothing else."""
    d = make(io, [100], 1, 2, 64, 32, seed=62)
    d["beta"][40] = 0.0
    clean = dict(d, v=d["v"].clone())
    clean["v"][40] = 0.0
    d["v"][40] = torch.finfo(DT[io]).min
    o, S = run_fwd(d)
    ref = want(clean, 64 ** -0.5, False)
    close(o, ref["o"], "o")
    close(S, ref["S"], "last_S")
