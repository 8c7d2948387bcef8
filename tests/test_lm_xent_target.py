"""bf16 gradients of the linear cross entropy hold g in bf16, but not what is as a rule most of a row's g: the
target's entry is made up for in dx and in dweight.  Against float64 on the GPU."""
import pytest
import torch

import lm_ref
from gpu_util import log
from test_lm_xent import inputs, ulp

pytestmark = pytest.mark.gpu


def half_step(v):
    """Half the distance of bf16 numbers around values of this size: 8 bits from the leading one on."""
    return torch.where(v > 0, torch.ldexp(torch.ones_like(v), torch.floor(torch.log2(v)).int() - 8), 0.0)


def inside(got, want, tol, what):
    got = got.detach().double().reshape(want.shape)
    assert torch.isfinite(got).all(), what
    bound = tol + half_step(want.abs() + tol)
    worst = float(((got - want).abs() / (bound + 1e-300)).max())
    log("  %s: %.3g of its bound" % (what, worst))
    assert worst <= 1, (what, worst)


def check(T, V, D, words=None, ignored=0.1, offset=0):
    import selective_state_space_msm_amd as msm
    gen = torch.Generator().manual_seed(T + V * 5 + D)
    x, w, t = inputs("bf16", T, V, D, ignored, gen, spread=0.5)
    if words:  # few words are targets: sums of many tokens
        t = torch.where((t >= 0) & (t < V), torch.tensor(words)[t % len(words)], t)
    log("T=%d V=%d D=%d" % (T, V, D))
    # 1 + 2^-8 is half way between bf16 numbers: g rounds by nearly the most there is, always to the same side
    dloss = torch.full((T,), 1.0039, device="cuda")
    xd, wd, t = x.double().cuda(), w.double().cuda(), t.cuda()
    _, lse, logits = lm_ref.xent_fwd(xd, wd, t, 1.0)
    lse = lse.float()
    gw = torch.empty(w.numel() + offset, dtype=w.dtype, device="cuda")[offset:].view(V, D).copy_(w)
    d = msm.msm_linear_cross_entropy_bwd(x.cuda(), gw, t, lse, dloss)
    g, p = lm_ref.xent_g(logits, t, lse.double(), dloss.double(), None, 1.0)
    # a logit: D products and their sum, 2^-24 each of the sum of sizes; p = exp(l - lse): that, the arguments'
    # roundings and the exponential's (test_lm_xent.check); g: its own roundings in fp32
    dl = ulp(D + 2) * (xd.abs() @ wd.abs().t())
    dg = p * (dl + ulp(4) * (logits.abs() + (logits - lse.double()[:, None]).abs()) + 2.0 ** -21) + ulp(4) * g.abs()
    del dl
    # every entry is rounded to bf16 once, the target's to twice that many bits
    live = (t >= 0) & (t < V)
    rounding = 2.0 ** -8 * (g.abs() + dg)
    rounding[live, t[live]] *= 2.0 ** -8
    dg += rounding
    dg += 3 * 2.0 ** -126
    ga = g.abs() + dg
    # sums of V (T) products, the target's once more
    tol = dg @ wd.abs() + ulp(V + 6) * (ga @ wd.abs())
    inside(d["dx"], g @ wd, tol, "dx")
    xa = torch.where(live[:, None], xd, 0.0).abs()
    tol = dg.t() @ xa + ulp(2 * T + 4) * (ga.t() @ xa)
    inside(d["dweight"], g.t() @ xd, tol, "dweight")


@pytest.mark.parametrize("T,V,D", [(1, 300, 64), (7, 1000, 40), (64, 64, 64), (130, 2500, 72), (512, 4099, 136)])
def test_rows_in_their_places(T, V, D):
    check(T, V, D)


@pytest.mark.parametrize("T,V,D", [(600, 1000, 64), (1030, 3001, 61), (2100, 8200, 1032), (700, 9000, 584), (2300, 40000, 520)])
def test_gathered_rows(T, V, D):
    """dweight in tiles of 64, 128 and 256."""
    check(T, V, D)


@pytest.mark.parametrize("T,V,D", [(4500, 40000, 72), (9000, 17000, 264), (9000, 1000, 64)])
def test_many_tokens(T, V, D):
    """More tokens than a workgroup looks at in one go, and more than one piece of the vocabulary."""
    check(T, V, D, ignored=0.02)


@pytest.mark.parametrize("T,V,D,words", [(32768, 700, 40, None), (32769, 700, 40, None), (40000, 9000, 72, None), (50000, 300, 520, None),
                                          (40000, 9000, 64, [0, 3327, 3328, 8999])])
def test_far_more_tokens(T, V, D, words):
    """Runs of up to 256 places, in one piece of the vocabulary and several."""
    check(T, V, D, words, ignored=0.02)


@pytest.mark.parametrize("T,V,D,words", [(400, 300, 64, [299]), (5000, 700, 72, [3]), (3000, 5000, 520, [0, 1, 17, 63, 64, 255, 256, 4999])])
def test_words_of_many_tokens(T, V, D, words):
    check(T, V, D, words)


def test_weights_copied_for_their_address():
    check(900, 3000, 136, offset=1)


def test_what_was_lost_in_other_calls_is_not_added():
    """A workspace of all kinds of bits, and rows that are left out in their places."""
    import selective_state_space_msm_amd as msm
    gen = torch.Generator().manual_seed(1)
    for T in (200, 700):
        x, w, t = (a.cuda() for a in inputs("bf16", T, 600, 72, 0.4, gen))
        lse = lm_ref.xent_fwd(x.double(), w.double(), t, 1.0)[1].float()
        dl = torch.full((T,), 1.0039, device="cuda")
        need = msm.msm_linear_cross_entropy_bwd_workspace_bytes(T, 600, 72, torch.bfloat16)
        got = [msm.msm_linear_cross_entropy_bwd(x, w, t, lse, dl, workspace=torch.full((need,), v, dtype=torch.uint8, device="cuda"))
               for v in (0, 255, 66)]
        for d in got[1:]:
            assert torch.equal(d["dx"], got[0]["dx"]) and torch.equal(d["dweight"], got[0]["dweight"])


@pytest.mark.parametrize("T,V", [(200, 700), (900, 3000), (4096, 900), (4097, 900), (5000, 60000)])
def test_captured_and_replayed(T, V):
    """Counting and sorting the targets in a graph: every replay on new inputs gives what a call of its own gives."""
    import selective_state_space_msm_amd as msm
    D = 72
    gen = torch.Generator().manual_seed(T)
    sets = []
    for _ in range(3):
        x, w, t = (a.cuda() for a in inputs("bf16", T, V, D, 0.2, gen))
        sets.append((x, w, t, msm.msm_linear_cross_entropy_fwd(x, w, t, return_lse=True)[1], torch.randn(T, generator=gen).cuda()))
    held = [a.clone() for a in sets[0]]
    ws = torch.full((msm.msm_linear_cross_entropy_bwd_workspace_bytes(T, V, D, torch.bfloat16),), 255, dtype=torch.uint8, device="cuda")
    out = {"dx": torch.empty_like(held[0]), "dweight": torch.empty_like(held[1])}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        msm.msm_linear_cross_entropy_bwd(*held, out=out, workspace=ws, stream=s)
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            msm.msm_linear_cross_entropy_bwd(*held, out=out, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for turn in range(6):
        now = sets[turn % 3]
        for a, b in zip(held, now):
            a.copy_(b)
        for a in out.values():
            a.fill_(float("nan"))
        want = msm.msm_linear_cross_entropy_bwd(*now)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["dx"], want["dx"]) and torch.equal(out["dweight"], want["dweight"]), turn
