"""Embedding, block norm and cross entropy in captured graphs: every replay gives what eager calls give."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def calls(msm, a, ws=None):
    """A training step's calls and a served token's; a holds their inputs."""
    e = msm.msm_embed_fwd(a["ids"], a["table"], 1.5, io=a["o"].dtype)
    r, y, rstd, q = msm.msm_block_norm_fwd(e, a["w"], a["o"], a["pw"], a["z"], 0.4, return_stats=True)
    loss, lse = msm.msm_linear_cross_entropy_fwd(y, a["head"], a["targets"], return_lse=True)
    x = msm.msm_linear_cross_entropy_bwd(y, a["head"], a["targets"], lse, a["dloss"], dlse=a["dlse"], workspace=ws)
    d = msm.msm_block_norm_bwd(r, x["dx"], rstd, a["w"], a["o"], q, a["pw"], a["z"], 0.4, dr_out=a["dr"])
    t = msm.msm_embed_bwd(a["ids"], d["dr"], a["table"].shape[0], 1.5, table_dtype=a["table"].dtype)
    served = msm.msm_linear_cross_entropy_fwd(y[:5].contiguous(), a["head"], a["targets"][:5].contiguous())
    return [e, r, y, rstd, q, loss, lse, *x.values(), *d.values(), t, served]


def inputs(io, T, V, D, seed):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    ids = torch.randint(-2, V, (T,), generator=gen)
    ids[: T // 3] = 3  # a busy row
    a = dict(ids=ids, table=rnd(V, D), o=rnd(T, D).to(io), z=rnd(T, D).to(io), w=1 + 0.1 * rnd(D), pw=1 + 0.1 * rnd(D),
             head=(rnd(V, D) * D ** -0.5).to(io), targets=torch.randint(-V // 4, V, (T,), generator=gen),
             dloss=rnd(T), dlse=0.1 * rnd(T), dr=rnd(T, D).to(io))
    return {n: t.cuda() for n, t in a.items()}


def capture(f):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()  # the library's code is loaded before the capture
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = f()
    return graph, got


@pytest.mark.parametrize("T,V,D", [(700, 900, 136), (5000, 300, 40), (40, 3000, 72)])
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_replays(io, T, V, D):
    import selective_state_space_msm_amd as msm
    a = inputs(io, T, V, D, 0)
    graph, got = capture(lambda: calls(msm, a))
    for seed in (1, 2, 3, 3):
        for n, t in inputs(io, T, V, D, seed).items():
            a[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        want = calls(msm, a)
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), (seed, i)


def test_two_graphs_in_turn():
    """Graphs with a workspace each may be replayed in any order; one that is the caller's own serves both when
    their replays do not overlap."""
    import selective_state_space_msm_amd as msm
    io = torch.bfloat16
    a, b = inputs(io, 300, 500, 64, 1), inputs(io, 300, 500, 64, 2)
    ws = torch.empty(msm.msm_linear_cross_entropy_bwd_workspace_bytes(300, 500, 64, io), dtype=torch.uint8, device="cuda")
    ga, xa = capture(lambda: calls(msm, a, ws))
    gb, xb = capture(lambda: calls(msm, b, ws))
    wa, wb = [t.clone() for t in calls(msm, a)], [t.clone() for t in calls(msm, b)]
    for g in (ga, gb, gb, ga, gb):
        g.replay()
    torch.cuda.synchronize()
    for got, want in ((xa, wa), (xb, wb)):
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), i
