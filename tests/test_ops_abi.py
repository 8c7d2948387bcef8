"""Refusals of the block operators: no GPU needed, nothing is launched."""
import ctypes

import pytest
import torch

import selective_state_space_msm_amd as msm

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    return msm.load_library()


def _delta(lib, bwd=False, **kw):
    a = dict(q=0x100000, k=0x200000, v=0x300000, g=0x400000, beta=0x500000, off=None, S0=None,
             do=0x600000, dl=None, o=0x1000000, lS=None, dq=0x2000000, dk=0x3000000, dv=0x4000000,
             dg=0x5000000, db=0x6000000, dS0=None, Bt=1, L=8, Hk=1, H=2, K=16, V=16, scale=1.0,
             io=0, ws=0x10000000, wsb=1 << 34)
    a.update(kw)
    sizes = [a[n] for n in ("Bt", "L", "Hk", "H", "K", "V")]
    tail = [ctypes.c_float(a["scale"]), a["io"], P(a["ws"]), a["wsb"], None]
    ins = [P(a[n]) for n in ("q", "k", "v", "g", "beta", "off", "S0")]
    if not bwd:
        return lib.msm_delta_rule_fwd(*ins, P(a["o"]), P(a["lS"]), *sizes, *tail)
    outs = [P(a[n]) for n in ("do", "dl", "dq", "dk", "dv", "dg", "db", "dS0")]
    return lib.msm_delta_rule_bwd(*ins, *outs, *sizes, *tail)


@pytest.mark.parametrize("bwd", [False, True])
def test_delta_refusals(lib, bwd):
    call = lambda **kw: _delta(lib, bwd, **kw)
    for n in ("q", "k", "v", "g", "beta") + (("do", "dq", "dk", "dv", "dg", "db") if bwd else ("o",)):
        assert call(**{n: None}) == INVALID, n
    for n in ("Bt", "L", "Hk", "H", "K", "V"):
        assert call(**{n: 0}) == INVALID, n
        assert call(**{n: -1}) == INVALID, n
    assert call(H=3, Hk=2) == INVALID
    assert call(K=257) == UNSUPPORTED
    assert call(io=2) == UNSUPPORTED
    assert call(H=65536) == INVALID
    assert call(L=1 << 31) == INVALID
    assert call(Bt=1 << 20, L=1 << 20) == INVALID
    assert call(scale=float("inf")) == INVALID
    assert call(scale=float("nan")) == INVALID
    assert call(ws=None) == WORKSPACE
    q = lib.msm_delta_rule_bwd_workspace_bytes if bwd else lib.msm_delta_rule_fwd_workspace_bytes
    need = q(1, 8, 1, 2, 16, 16, 0, 0)
    assert need > 0 and call(wsb=need - 1) == WORKSPACE
    assert call(ws=0x10000004) == INVALID
    out = "dv" if bwd else "o"
    assert call(**{out: 0x300000}) == INVALID
    assert call(**{out: 0x100010}) == INVALID
    assert call(S0=0x700000, **{"dS0" if bwd else "lS": 0x700000}) == INVALID
    assert call(off=0x10000010) == INVALID  # inside the workspace

@pytest.mark.parametrize("bwd", [False, True])
def test_delta_refuses_rows_past_32_bit_offsets(lib, bwd):
    """64 rows of 2^18 x 32 fp32 values are 2^31 bytes, of bf16 ones half of that."""
    q = lib.msm_delta_rule_bwd_workspace_bytes if bwd else lib.msm_delta_rule_fwd_workspace_bytes
    wide = dict(Hk=1, H=32, K=16, V=1 << 18)
    assert _delta(lib, bwd, **wide) == UNSUPPORTED
    assert q(1, 8, 1, 32, 16, 1 << 18, 0, 0) == 0
    assert q(1, 8, 1, 32, 16, 1 << 18, 0, 1) > 0
    assert _delta(lib, bwd, V=(1 << 20) + 1) == INVALID
    assert q(1, 8, 1, 65535, 16, 1 << 20, 0, 1) == 0



@pytest.mark.parametrize("bwd", [False, True])
def test_delta_refuses_launches_past_32_bits(lib, bwd):
    """A launch has fewer than 2^32 threads: 2^24 workgroups of 256, one a chunk or a sequence and head."""
    q = lib.msm_delta_rule_bwd_workspace_bytes if bwd else lib.msm_delta_rule_fwd_workspace_bytes
    for sizes, packed in (((1 << 24, 1, 1, 1, 16, 16), 0), ((1 << 15, 1, 1, 512, 16, 16), 0),
                          ((1 << 15, 4, 1, 512, 16, 16), 1), ((1, (1 << 30) + 64, 1, 1, 16, 16), 1)):
        a = dict(zip(("Bt", "L", "Hk", "H", "K", "V"), sizes), wsb=1 << 62)
        # arrays of such sizes do not overlap only if they are far apart
        places = ["q", "k", "v", "g", "beta", "do", "o", "dq", "dk", "dv", "dg", "db", "ws"]
        a.update({n: (i + 1) << 48 for i, n in enumerate(places)})
        if packed:
            a["off"] = 1 << 20
        assert _delta(lib, bwd, **a) == UNSUPPORTED, sizes
        assert q(*sizes, packed, 0) == 0
    assert q((1 << 24) - 64, 1, 1, 1, 16, 16, 0, 0) > 0
    step = [P((i + 1) << 40) for i in range(7)]
    step[0] = None  # refused for this, not for its 2^24 states
    assert lib.msm_delta_rule_step(*step, 1 << 24, 1, 1, 16, 16, ctypes.c_float(1), 0, None) == INVALID


def test_delta_workspace_queries(lib):
    for q in (lib.msm_delta_rule_fwd_workspace_bytes, lib.msm_delta_rule_bwd_workspace_bytes):
        assert q(0, 8, 1, 1, 16, 16, 0, 0) == 0
        assert q(1, 8, 2, 3, 16, 16, 0, 0) == 0
        assert q(1, 8, 1, 1, 300, 16, 0, 0) == 0
        assert q(1, 8, 1, 1, 16, 16, 0, 9) == 0
        # a packed batch has a chunk for every started 64 tokens of each of its sequences at most
        assert q(4, 256, 1, 1, 16, 16, 1, 0) >= q(1, 256, 1, 1, 16, 16, 0, 0)


def test_step_refusals(lib):
    def call(**kw):
        a = dict(q=0x100000, k=0x200000, v=0x300000, g=0x400000, beta=0x500000, S=0x1000000, o=0x2000000,
                 Bt=1, Hk=1, H=2, K=16, V=16, scale=1.0, io=0)
        a.update(kw)
        return lib.msm_delta_rule_step(*(P(a[n]) for n in ("q", "k", "v", "g", "beta", "S", "o")),
                                       *(a[n] for n in ("Bt", "Hk", "H", "K", "V")),
                                       ctypes.c_float(a["scale"]), a["io"], None)

    for n in ("q", "k", "v", "g", "beta", "S", "o"):
        assert call(**{n: None}) == INVALID, n
    for n in ("Bt", "Hk", "H", "K", "V"):
        assert call(**{n: 0}) == INVALID, n
    assert call(K=257) == UNSUPPORTED
    assert call(io=5) == UNSUPPORTED
    assert call(H=3, Hk=2) == INVALID
    assert call(S=0x300000) == INVALID
    assert call(o=0x1000000) == INVALID
    assert call(scale=float("nan")) == INVALID


def test_norm_refusals(lib):
    def fwd(**kw):
        a = dict(x=0x100000, w=None, b=None, y=0x200000, mean=None, rstd=None, rows=4, D=32, eps=1e-5, io=0)
        a.update(kw)
        return lib.msm_layer_norm_fwd(*(P(a[n]) for n in ("x", "w", "b", "y", "mean", "rstd")), a["rows"],
                                      a["D"], ctypes.c_float(a["eps"]), a["io"], None)

    def bwd(**kw):
        a = dict(x=0x100000, w=0x110000, dy=0x120000, mean=0x130000, rstd=0x140000, dx=0x200000,
                 dw=0x210000, db=0x220000, rows=4, D=32, io=0, ws=0x1000000, wsb=1 << 30)
        a.update(kw)
        return lib.msm_layer_norm_bwd(*(P(a[n]) for n in ("x", "w", "dy", "mean", "rstd", "dx", "dw", "db")),
                                      a["rows"], a["D"], a["io"], P(a["ws"]), a["wsb"], None)

    for f, ptrs in ((fwd, ("x", "y")), (bwd, ("x", "dy", "mean", "rstd", "dx"))):
        for n in ptrs:
            assert f(**{n: None}) == INVALID, n
        assert f(rows=0) == INVALID and f(D=0) == INVALID and f(rows=-2) == INVALID
        assert f(rows=1 << 31) == INVALID and f(D=(1 << 30) + 1) == INVALID
        assert f(io=3) == UNSUPPORTED
    assert fwd(eps=-1.0) == INVALID and fwd(eps=float("nan")) == INVALID and fwd(eps=float("inf")) == INVALID
    assert fwd(y=0x100000) == INVALID
    assert bwd(dx=0x120000) == INVALID
    assert bwd(ws=None) == WORKSPACE and bwd(wsb=8) == WORKSPACE and bwd(ws=0x1000008) == INVALID
    assert lib.msm_layer_norm_bwd_workspace_bytes(0, 4, 0) == 0


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("rows,D", [(1, 1 << 28), (3, 5001), (1, 4096), (7, 16)])
def test_norm_workspace_of_few_rows(lib, rows, D, io):
    """A pair of column sums for every workgroup, and no more workgroups than rows."""
    assert lib.msm_layer_norm_bwd_workspace_bytes(rows, D, io) <= rows * 8 * D + 256


def test_clip_refusals(lib):
    def call(clip=True, src=(0x100000, 0x200000), dst=None, n=(16, 16), t=(0, 1), count=2, norm=0x300000,
             ws=0x1000000, wsb=1 << 20, max_norm=1.0, eps=1e-6):
        k = len(src)
        a = (P * k)(*src)
        d = None if dst is None else (P * k)(*dst)
        nn, tt = (ctypes.c_int64 * k)(*n), (ctypes.c_int32 * k)(*t)
        if clip:
            return lib.msm_grad_clip(a, d, nn, tt, count, ctypes.c_float(max_norm), ctypes.c_float(eps), P(norm),
                                     P(ws), wsb, None)
        return lib.msm_grad_norm(a, nn, tt, count, P(norm), P(ws), wsb, None)

    for clip in (False, True):
        assert call(clip, count=-1) == INVALID
        assert call(clip, n=(16, -1)) == INVALID
        assert call(clip, src=(0x100000, None)) == INVALID
        assert call(clip, src=(0x100002, 0x200000)) == INVALID  # an fp32 tensor off its elements
        assert call(clip, t=(0, 2)) == UNSUPPORTED
        assert call(clip, norm=None) == INVALID
        assert call(clip, ws=None) == WORKSPACE
        assert call(clip, wsb=64) == WORKSPACE
        assert call(clip, ws=0x1000004) == INVALID
    assert call(max_norm=-1.0) == INVALID and call(max_norm=float("nan")) == INVALID
    assert call(eps=-1.0) == INVALID
    assert call(dst=(0x100004, 0x400000)) == INVALID  # overlapping its own gradient
    assert call(dst=(None, 0x400000)) == INVALID
    assert lib.msm_grad_norm_workspace_bytes(-1) == 0
    assert lib.msm_grad_norm(None, None, None, 1, P(1), P(16), 1 << 20, None) == INVALID


def test_clip_refuses_overlaps(lib):
    """Each of these would let a write reach what another part of the call reads or writes."""
    def call(clip, src, dst=None, n=16, norm=0x300000, ws=0x1000000):
        k = len(src)
        a, d = (P * k)(*src), None if dst is None else (P * k)(*dst)
        nn, tt = (ctypes.c_int64 * k)(*([n] * k)), (ctypes.c_int32 * k)()
        if clip:
            return lib.msm_grad_clip(a, d, nn, tt, k, ctypes.c_float(1), ctypes.c_float(0), P(norm), P(ws), 1 << 20, None)
        return lib.msm_grad_norm(a, nn, tt, k, P(norm), P(ws), 1 << 20, None)

    two = (0x100000, 0x200000)
    assert call(True, two, dst=(0x200000, 0x400000)) == INVALID  # another gradient
    assert call(True, two, dst=(0x400000, 0x100020)) == INVALID  # inside another gradient
    assert call(True, two, dst=(0x100000, 0x100000)) == INVALID  # in place, and then again
    assert call(True, two, dst=(0x400000, 0x400020)) == INVALID  # another output
    assert call(True, two, dst=(0x400000, 0x300000)) == INVALID  # the norm
    assert call(True, two, dst=(0x400000, 0x1000100)) == INVALID  # the workspace
    assert call(True, (0x100000, 0x200000, 0x100000)) == INVALID  # one gradient twice, in place
    assert call(True, (0x100000, 0x100020)) == INVALID            # two that share elements, in place
    many = [0x40000000 + 0x100 * i for i in range(3000)]
    assert call(True, many[::-1] + [many[1700]]) == INVALID
    assert call(True, many, dst=[x + (1 << 40) for x in many[:-1]] + [many[7]]) == INVALID
    for clip in (False, True):
        assert call(clip, (0x100000, 0x300000 - 60)) == INVALID   # the norm in a gradient
        assert call(clip, (0x100000, 0x1000000)) == INVALID       # the workspace in a gradient
        assert call(clip, two, norm=0x1000008) == INVALID         # the norm in the workspace


def test_python_refusals():
    """Shapes, dtypes and strides are refused before the library is called (CPU tensors serve)."""
    q, v = torch.zeros(1, 4, 1, 8), torch.zeros(1, 4, 2, 8)
    g = torch.zeros(1, 4, 2)
    f = msm.msm_delta_rule_fwd
    with pytest.raises(ValueError, match="k has shape"):
        f(q, q[:, :3], v, g, g)
    with pytest.raises(ValueError, match="contiguous"):
        f(q, q, v.transpose(2, 3), g, g)
    with pytest.raises(ValueError, match="dtype"):
        f(q, q, v.bfloat16(), g, g)
    with pytest.raises(ValueError, match="g has dtype"):
        f(q, q, v, g.double(), g)
    with pytest.raises(ValueError, match="unsupported io dtype"):
        f(q.half(), q.half(), v.half(), g, g)
    with pytest.raises(ValueError, match="shapes"):
        f(q[0], q[0], v[0], g[0], g[0])
    with pytest.raises(ValueError, match="seq_offsets"):
        f(q[0], q[0], v[0], g[0], g[0], seq_offsets=torch.zeros(3))
    with pytest.raises(ValueError, match="S has shape"):
        msm.msm_delta_rule_step(q[0], q[0], v[0], g[0], g[0], torch.zeros(4, 2, 8, 7))
    with pytest.raises(ValueError, match="weight"):
        msm.msm_layer_norm_fwd(torch.zeros(3, 8), torch.zeros(7))
    with pytest.raises(ValueError, match="mean"):
        msm.msm_layer_norm_bwd(torch.zeros(3, 8), torch.zeros(3, 8), torch.zeros(2), torch.zeros(3))
    with pytest.raises(ValueError, match="no gradients"):
        msm.msm_grad_norm([])
    with pytest.raises(ValueError, match="contiguous"):
        msm.msm_grad_clip([torch.zeros(4, 5).t()], 1.0)
    with pytest.raises(ValueError, match="unsupported dtype"):
        msm.msm_grad_norm([torch.zeros(4, dtype=torch.float64)])
    with pytest.raises(ValueError, match="differs"):
        msm.msm_grad_clip([torch.zeros(4)], 1.0, out=[torch.zeros(5)])


class _Stream:
    """Enough of a stream for a call that must be refused before it uses one."""
    cuda_stream = 0
    device = torch.device("cuda", 0)


def test_host_tensors_are_refused_on_a_given_stream():
    q, v, g = torch.zeros(1, 4, 1, 8), torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2)
    x, m = torch.zeros(3, 8), torch.zeros(3)
    s = _Stream()
    outs = {n: torch.zeros(shape) for n, shape in (("dq", q.shape), ("dk", q.shape), ("dv", v.shape), ("dg", g.shape),
                                                   ("dbeta", g.shape))}
    calls = [
        lambda: msm.msm_delta_rule_fwd(q, q, v, g, g, stream=s),
        lambda: msm.msm_delta_rule_bwd(q, q, v, g, g, v, stream=s, out=outs),
        lambda: msm.msm_delta_rule_step(q[0], q[0], v[0], g[0], g[0], torch.zeros(4, 2, 8, 8), stream=s),
        lambda: msm.msm_layer_norm_fwd(x, stream=s),
        lambda: msm.msm_layer_norm_bwd(x, x, m, m, stream=s),
        lambda: msm.msm_grad_norm([x], stream=s),
        lambda: msm.msm_grad_clip([x], 1.0, stream=s),
        lambda: msm.msm_scan_fwd(torch.zeros(1, 4, 8), torch.zeros(1, 4, 8), torch.zeros(8, 4), torch.zeros(1, 4, 4),
                                 torch.zeros(1, 4, 4), 0.9, 1.0, stream=s),
    ]
    for f in calls:
        with pytest.raises(ValueError, match="on a GPU"):
            f()


def test_workspace_is_checked():
    """As the other arguments are: where it lies and how (meta tensors stand for another device's)."""
    from selective_state_space_msm_amd import _Owned, _workspace
    own, cpu = _Owned(None), torch.device("cpu")
    with pytest.raises(ValueError, match="workspace is on meta"):
        _workspace(64, torch.empty(64, dtype=torch.uint8, device="meta"), cpu, own)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        _workspace(64, torch.zeros(128, dtype=torch.uint8)[::2], cpu, own)
    with pytest.raises(msm.MsmError):
        _workspace(64, torch.zeros(63, dtype=torch.uint8), cpu, own)
    assert _workspace(64, torch.zeros(16), cpu, own)[1] == 64
    assert _workspace(0, None, cpu, own) == (None, 0)
