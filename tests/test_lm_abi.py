"""Refusals of the embedding, the block norm and the linear cross entropy: no GPU needed, nothing is launched."""
import ctypes

import pytest
import torch

import selective_state_space_msm_amd as msm

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P, F = ctypes.c_void_p, ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    return msm.load_library()


def embed(lib, bwd, **kw):
    a = dict(ids=0x100000, a=0x200000, y=0x1000000, T=8, V=9, D=16, scale=1.0, table=0, io=0, ws=0x10000000, wsb=1 << 34)
    a.update(kw)
    args = [P(a["ids"]), P(a["a"]), P(a["y"]), a["T"], a["V"], a["D"], F(a["scale"]), a["table"], a["io"]]
    if bwd:
        return lib.msm_embed_bwd(*args, P(a["ws"]), a["wsb"], None)
    return lib.msm_embed_fwd(*args, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_embed_refusals(lib, bwd):
    call = lambda **kw: embed(lib, bwd, **kw)
    for n in ("ids", "a", "y"):
        assert call(**{n: None}) == INVALID, n
    for n in ("T", "V", "D"):
        assert call(**{n: 0}) == INVALID and call(**{n: -1}) == INVALID, n
    assert call(T=1 << 31) == INVALID and call(V=(1 << 31) - 1) == INVALID and call(D=(1 << 24) + 1) == INVALID
    assert call(table=2) == UNSUPPORTED and call(io=-1) == UNSUPPORTED
    assert call(scale=float("nan")) == INVALID and call(scale=float("inf")) == INVALID
    assert call(ids=0x100004) == INVALID
    assert call(a=0x200002) == INVALID and call(y=0x1000001, table=1, io=1) == INVALID
    assert call(y=0x100000) == INVALID and call(y=0x200010) == INVALID
    if bwd:
        need = lib.msm_embed_bwd_workspace_bytes(8, 9, 16)
        assert need > 0 and call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
        assert call(ws=0x10000008) == INVALID and call(ws=0x1000000) == INVALID
    assert lib.msm_embed_bwd_workspace_bytes(0, 9, 16) == 0


def norm(lib, bwd, **kw):
    a = dict(r=0x1000000, w=0x100000, o=0x2000000, pw=0x110000, z=0x3000000, ro=0x4000000, y=0x5000000, rs=0x120000, prs=0x130000,
             dro=0x6000000, dr=0x7000000, do=0x8000000, dz=0x9000000, dw=0x140000, dpw=0x150000, rows=8, D=64, scale=1.0,
             eps=1e-5, io=0, ws=0x10000000, wsb=1 << 34)
    a.update(kw)
    p = lambda *n: [P(a[i]) for i in n]
    if bwd:
        return lib.msm_block_norm_bwd(*p("ro", "y", "rs", "w", "o", "prs", "pw", "z", "dro", "dr", "do", "dz", "dw", "dpw"),
                                      a["rows"], a["D"], F(a["scale"]), a["io"], P(a["ws"]), a["wsb"], None)
    return lib.msm_block_norm_fwd(*p("r", "w", "o", "pw", "z", "ro", "y", "rs", "prs"), a["rows"], a["D"], F(a["scale"]),
                                  F(a["eps"]), a["io"], None)


@pytest.mark.parametrize("bwd", [False, True])
def test_block_norm_refusals(lib, bwd):
    call = lambda **kw: norm(lib, bwd, **kw)
    for n in ("ro", "y", "rs", "dr", "do", "prs") if bwd else ("r", "y", "ro"):
        assert call(**{n: None}) == INVALID, n
    for n in ("rows", "D"):
        assert call(**{n: 0}) == INVALID and call(**{n: -1}) == INVALID, n
    assert call(rows=1 << 31) == INVALID and call(D=(1 << 30) + 1) == INVALID and call(rows=1 << 30, D=1 << 30) == INVALID
    assert call(io=2) == UNSUPPORTED
    assert call(scale=float("nan")) == INVALID
    # what belongs to the block without the block
    assert call(o=None) == INVALID
    if bwd:
        gone = dict(o=None, prs=None, pw=None, z=None, do=None, dz=None, dpw=None)
        for n in ("prs", "pw", "z", "do", "dz", "dpw"):
            assert call(**{**gone, n: 0xA000000}) == INVALID, n
        assert call(z=None) == INVALID and call(dz=None) == INVALID
        need = lib.msm_block_norm_bwd_workspace_bytes(8, 64, 0)
        assert need > 0 and call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
        assert call(ws=0x10000008) == INVALID
        assert call(dr=0x4000000) == INVALID and call(do=0x7000010) == INVALID and call(dpw=0x140000) == INVALID
        assert call(dr=0x7000002) == INVALID
    else:
        gone = dict(o=None, pw=None, z=None, ro=None, prs=None)
        for n in ("pw", "z", "ro", "prs"):
            assert call(**{**gone, n: 0xA000000}) == INVALID, n
        assert call(eps=-1.0) == INVALID and call(eps=float("inf")) == INVALID and call(eps=float("nan")) == INVALID
        assert call(y=0x1000000) == INVALID and call(ro=0x1000010) == INVALID and call(ro=0x2000000) == INVALID
        assert call(y=0x4000000) == INVALID and call(y=0x5000001, io=1) == INVALID
    assert lib.msm_block_norm_bwd_workspace_bytes(8, 0, 0) == 0


def xent(lib, bwd, **kw):
    a = dict(x=0x1000000, w=0x2000000, t=0x100000, loss=0x110000, lse=0x120000, dloss=0x130000, dlse=0x140000, dx=0x3000000,
             dw=0x4000000, T=8, V=100, D=32, scale=1.0, io=0, ws=0x40000000, wsb=1 << 34)
    a.update(kw)
    p = lambda *n: [P(a[i]) for i in n]
    tail = [a["T"], a["V"], a["D"], F(a["scale"]), a["io"], P(a["ws"]), a["wsb"], None]
    if bwd:
        return lib.msm_linear_cross_entropy_bwd(*p("x", "w", "t", "lse", "dloss", "dlse", "dx", "dw"), *tail)
    return lib.msm_linear_cross_entropy_fwd(*p("x", "w", "t", "loss", "lse"), *tail)


@pytest.mark.parametrize("bwd", [False, True])
def test_xent_refusals(lib, bwd):
    call = lambda **kw: xent(lib, bwd, **kw)
    for n in ("x", "w", "t", "lse", "dloss", "dx") if bwd else ("x", "w", "t", "loss"):
        assert call(**{n: None}) == INVALID, n
    for n in ("T", "V", "D"):
        assert call(**{n: 0}) == INVALID and call(**{n: -1}) == INVALID, n
    assert call(T=(1 << 22) + 1) == UNSUPPORTED and call(V=(1 << 22) + 1) == UNSUPPORTED and call(D=(1 << 16) + 1) == UNSUPPORTED
    assert call(T=1 << 19, V=(1 << 18) + 1, wsb=1 << 60) == UNSUPPORTED
    assert call(io=3) == UNSUPPORTED
    assert call(scale=float("inf")) == INVALID
    assert call(t=0x100004) == INVALID and call(x=0x1000002) == INVALID and call(w=0x2000001, io=1) == INVALID
    q = lib.msm_linear_cross_entropy_bwd_workspace_bytes if bwd else lib.msm_linear_cross_entropy_fwd_workspace_bytes
    need = q(8, 100, 32, 0)
    assert need > 0 and call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    assert call(ws=0x40000008) == INVALID and call(ws=0x1000000) == INVALID
    assert q(8, 100, 0, 0) == 0 and q(8, 100, 32, 5) == 0
    if bwd:
        assert call(dx=0x1000000) == INVALID and call(dw=0x2000010) == INVALID and call(dx=0x4000000) == INVALID
        assert call(dx=0x120000) == INVALID and call(dw=0x4000002) == INVALID
    else:
        assert call(loss=0x120000) == INVALID and call(lse=0x100000) == INVALID and call(loss=0x1000000) == INVALID


def test_binding_refuses():
    """Shapes, types and places are checked before the library is called; tensors here are on the CPU."""
    ids, table, x = torch.zeros(4, dtype=torch.int64), torch.zeros(5, 8), torch.zeros(4, 8)
    one = torch.zeros(4)
    for call in (
        lambda: msm.msm_embed_fwd(ids.int(), table),
        lambda: msm.msm_embed_fwd(ids, table.half()),
        lambda: msm.msm_embed_fwd(ids, table[:, ::2]),
        lambda: msm.msm_embed_fwd(ids, table[0]),
        lambda: msm.msm_embed_fwd(ids, table, y=torch.zeros(4, 7)),
        lambda: msm.msm_embed_fwd(ids, table),                      # not on a GPU
        lambda: msm.msm_embed_bwd(ids, x[:3], 5),
        lambda: msm.msm_embed_bwd(ids, x[0], 5),
        lambda: msm.msm_embed_bwd(ids, x, 5, dtable=torch.zeros(4, 8)),
        lambda: msm.msm_block_norm_fwd(x, one),
        lambda: msm.msm_block_norm_fwd(x[0, 0]),
        lambda: msm.msm_block_norm_bwd(x[0, 0], x[0, 0], one),
        lambda: msm.msm_block_norm_fwd(x, None, None, torch.ones(8)),
        lambda: msm.msm_block_norm_fwd(x, None, None, None, x),
        lambda: msm.msm_block_norm_fwd(x, None, x.bfloat16()),
        lambda: msm.msm_block_norm_fwd(x, None, x, r_out=torch.zeros(4, 8).t()),
        lambda: msm.msm_block_norm_fwd(x, None, r_out=torch.zeros(4, 8)),
        lambda: msm.msm_block_norm_bwd(x, x, one, None, x),
        lambda: msm.msm_block_norm_bwd(x, x, one, None, None, one),
        lambda: msm.msm_block_norm_bwd(x, x[:3], one),
        lambda: msm.msm_linear_cross_entropy_fwd(x, table, ids.int()),
        lambda: msm.msm_linear_cross_entropy_fwd(x, table.bfloat16(), ids),
        lambda: msm.msm_linear_cross_entropy_fwd(x[:3], table, ids),
        lambda: msm.msm_linear_cross_entropy_fwd(x, table, ids, loss=torch.zeros(3)),
        lambda: msm.msm_linear_cross_entropy_bwd(x, table, ids, one, one.double()),
        lambda: msm.msm_linear_cross_entropy_bwd(x, table, ids, one, one, out={"dx": torch.zeros(4, 9)}),
        lambda: msm.msm_linear_cross_entropy_bwd(x, table, ids, one, one),
    ):
        with pytest.raises((ValueError, TypeError, msm.MsmError)):
            call()
