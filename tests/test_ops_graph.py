"""The block operators in a captured graph: every replay gives what eager calls give."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def eager(msm, a):
    """A training step's calls and two served tokens; a holds their inputs."""
    y, mean, rstd = msm.msm_layer_norm_fwd(a["x"], a["w"], a["b"], return_stats=True)
    v = y.view(a["x"].shape[:-1] + (4, 32))
    o, S = msm.msm_delta_rule_fwd(a["q"], a["k"], v, a["g"], a["beta"], return_last_state=True, **a["where"])
    d = msm.msm_delta_rule_bwd(a["q"], a["k"], v, a["g"], a["beta"], a["do"], **a["where"])
    n = msm.msm_layer_norm_bwd(a["x"], d["dv"].view(a["x"].shape), mean, rstd, a["w"], bias_grad=True)
    grads = [n["dweight"], n["dbias"], d["dq"], d["dk"]]
    clipped = [torch.empty_like(t) for t in grads]
    norm = msm.msm_grad_clip(grads, 0.5, out=clipped)
    S = S[:1].clone()
    tokens = [msm.msm_delta_rule_step(*(a[m][t].contiguous() for m in ("sq", "sk", "sv", "sg", "sb")), S)
              for t in range(2)]
    return [y, o, *d.values(), n["dx"], *grads, *clipped, norm, S, *tokens]


def inputs(io, packed, seed):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    lead = (900,) if packed else (2, 700)
    a = dict(x=rnd(*lead, 128).to(io), q=rnd(*lead, 2, 32).to(io), k=(rnd(*lead, 2, 32) * 32 ** -0.5).to(io),
             do=rnd(*lead, 4, 32).to(io), g=-torch.rand(*lead, 4, generator=gen),
             beta=torch.rand(*lead, 4, generator=gen), w=1 + 0.1 * rnd(128), b=rnd(128),
             sq=rnd(2, 1, 2, 32).to(io), sk=(rnd(2, 1, 2, 32) * 32 ** -0.5).to(io), sv=rnd(2, 1, 4, 32).to(io),
             sg=-torch.rand(2, 1, 4, generator=gen), sb=torch.rand(2, 1, 4, generator=gen))
    return {n: t.cuda() for n, t in a.items()}


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_replays(io, packed):
    import selective_state_space_msm_amd as msm
    a = inputs(io, packed, 0)
    where = {}
    if packed:
        where["seq_offsets"] = torch.tensor([0, 0, 130, 131, 900], dtype=torch.int32, device="cuda")
    a["where"] = where
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager(msm, a)  # the library's code is loaded before the capture
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = eager(msm, a)
    for seed in (1, 2, 3, 3):
        for n, t in inputs(io, packed, seed).items():
            a[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        want = eager(msm, a)
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), (seed, i)
