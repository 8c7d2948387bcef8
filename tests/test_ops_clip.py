"""Gradient norm and clipping on the GPU against float64."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SIZES = [0, 1, 3, 255, 2048, 2049, 16384, 16385, 100003]


def make(count, seed=0, scale=0.1, mixed=True, offset=False):
    gen = torch.Generator().manual_seed(seed)
    out = []
    for i in range(count):
        n = SIZES[i % len(SIZES)]
        dt = torch.bfloat16 if mixed and i % 2 else torch.float32
        buf = torch.empty(n + 1, dtype=dt, device="cuda")
        t = buf[1:] if offset else buf[:n]
        t.copy_(scale * torch.randn(n, generator=gen))
        out.append(t)
    return out


def exact_norm(grads):
    return sum(float(t.double().square().sum()) for t in grads) ** 0.5


@pytest.mark.parametrize("count", [1, 2, 9, 96, 97, 300])
@pytest.mark.parametrize("offset", [False, True])
def test_norm_and_clip(count, offset):
    import selective_state_space_msm_amd as msm
    grads = make(count, seed=count, offset=offset)
    want = exact_norm(grads)
    norm = msm.msm_grad_norm(grads)
    # one rounding of the sum's root to fp32
    assert abs(float(norm) - want) <= 1e-7 * want + 1e-30
    for max_norm in (0.5 * want, 2 * want + 1):
        coef = min(1.0, max_norm / (want + 1e-6))
        out = [torch.full_like(t, 9.0) for t in grads]
        n = msm.msm_grad_clip(grads, max_norm, out=out)
        assert float(n) == float(norm)
        for t, o in zip(grads, out):
            ref = t.double() * coef
            # two roundings of the factor and one of the product; bf16 rounds once more
            tol = 3e-7 if t.dtype == torch.float32 else 2.0 ** -8
            assert bool(((o.double() - ref).abs() <= tol * ref.abs()).all())
            if coef == 1.0:
                assert torch.equal(o, t)
    # in place, the same bits
    out = [torch.empty_like(t) for t in grads]
    msm.msm_grad_clip(grads, 0.25 * want, out=out)
    msm.msm_grad_clip(grads, 0.25 * want)
    for t, o in zip(grads, out):
        assert torch.equal(t, o)


def test_all_empty():
    import selective_state_space_msm_amd as msm
    grads = [torch.empty(0, device="cuda"), torch.empty(0, device="cuda", dtype=torch.bfloat16)]
    assert float(msm.msm_grad_norm(grads)) == 0.0
    assert float(msm.msm_grad_clip(grads, 1.0)) == 0.0


def test_huge_and_tiny_values():
    import selective_state_space_msm_amd as msm
    for scale in (1e30, 1e-30):
        g = [torch.full((5000,), scale, device="cuda"), torch.full((77,), scale, device="cuda")]
        want = scale * 5077 ** 0.5
        assert abs(float(msm.msm_grad_norm(g)) - want) <= 2e-7 * want


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite(bad):
    import selective_state_space_msm_amd as msm
    g = [torch.ones(3000, device="cuda"), torch.ones(10, device="cuda", dtype=torch.bfloat16)]
    g[0][1234] = bad
    norm = float(msm.msm_grad_clip(g, 1.0))
    if bad != bad:
        assert norm != norm and bool(torch.isnan(g[0]).all()) and bool(torch.isnan(g[1]).all())
    else:
        assert norm == bad and bool((g[1] == 0).all())


def test_zero_max_norm_and_repeat():
    import selective_state_space_msm_amd as msm
    g = make(20, seed=3)
    a, b = [torch.empty_like(t) for t in g], [torch.empty_like(t) for t in g]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    n1 = msm.msm_grad_clip(g, 0.3, out=a)
    n2 = msm.msm_grad_clip(g, 0.3, out=b, stream=s)
    torch.cuda.synchronize()
    assert float(n1) == float(n2)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    msm.msm_grad_clip(g, 0.0)
    assert all(bool((t == 0).all()) for t in g)


def test_graph_replays():
    """Captured in a graph and replayed between eager calls: every replay equals the eager result."""
    import selective_state_space_msm_amd as msm
    g = make(120, seed=5)
    out = [torch.empty_like(t) for t in g]
    ws = torch.empty(msm.msm_grad_norm_workspace_bytes(len(g)), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    msm.msm_grad_clip(g, 0.5, out=out, workspace=ws, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = msm.msm_grad_clip(g, 0.5, out=out, workspace=ws)
    for i in range(3):
        for t in g:
            t.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        got, n = [o.clone() for o in out], float(norm)
        ref = [torch.empty_like(t) for t in g]
        assert float(msm.msm_grad_clip(g, 0.5, out=ref)) == n
        assert all(torch.equal(x, y) for x, y in zip(got, ref))


def test_very_many_tensors():
    """The join of the partial sums happens once, not again in every scaling launch: with as many
    launches as the sums took, clipping takes about twice the norm's time.  (Joined in each of the
    2048 launches here, clipping took over ten times as long.)"""
    import ctypes
    import selective_state_space_msm_amd as msm
    lib = msm.load_library()
    count = 1 << 18
    src = torch.randn(count, device="cuda")
    out = torch.empty_like(src)
    P = ctypes.c_void_p
    addresses = lambda t: (P * count)(*range(t.data_ptr(), t.data_ptr() + 4 * count, 4))
    a, b = addresses(src), addresses(out)
    n, kind = (ctypes.c_int64 * count)(*[1] * count), (ctypes.c_int32 * count)()
    norm = torch.empty((), device="cuda")
    ws = torch.empty(msm.msm_grad_norm_workspace_bytes(count), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream()
    tail = (P(norm.data_ptr()), P(ws.data_ptr()), ws.numel(), P(stream.cuda_stream))

    def seconds(f):
        best = float("inf")
        for _ in range(3):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda.synchronize()
            start.record()
            assert f() == 0
            end.record()
            torch.cuda.synchronize()
            best = min(best, start.elapsed_time(end) * 1e-3)
        return best

    t_norm = seconds(lambda: lib.msm_grad_norm(a, n, kind, count, *tail))
    want = float(src.double().norm())
    assert abs(float(norm) - want) <= 1e-7 * want
    f = ctypes.c_float
    t_clip = seconds(lambda: lib.msm_grad_clip(a, b, n, kind, count, f(0.5 * want), f(0.0), *tail))
    assert abs(float(norm) - want) <= 1e-7 * want
    assert bool(((out - 0.5 * src).abs() <= 3e-7 * src.abs()).all())
    print("norm %.4f s, clipping %.4f s" % (t_norm, t_clip))
    assert t_clip <= 5 * t_norm, (t_clip, t_norm)
