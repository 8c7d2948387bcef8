"""Python binding of the operators at a language model's ends and between its blocks: token
embedding, the norms around a block with its gate and residual scale, and the cross entropy of a
linear layer over a vocabulary.  Same manner as the scan's binding: names of the C entry points,
argument checks and marshalling only, every step in the library's HIP kernels.

    x = msm_embed_fwd(ids, table, scale)                                        # (..., D)
    dtable = msm_embed_bwd(ids, dx, V, scale)
    r, y = msm_block_norm_fwd(r, weight, o, post_weight, z, scale)              # r' and the next block's input
    grads = msm_block_norm_bwd(r, dy, rstd, weight, o, post_rstd, post_weight, z, scale, dr_out=dr)
    loss, lse = msm_linear_cross_entropy_fwd(y, head, targets, return_lse=True)
    grads = msm_linear_cross_entropy_bwd(y, head, targets, lse, dloss)          # dx, dweight
"""
from __future__ import annotations

import ctypes

__all__ = [
    "msm_embed_fwd", "msm_embed_bwd", "msm_embed_bwd_workspace_bytes", "msm_block_norm_fwd",
    "msm_block_norm_bwd", "msm_block_norm_bwd_workspace_bytes", "msm_linear_cross_entropy_fwd",
    "msm_linear_cross_entropy_fwd_workspace_bytes", "msm_linear_cross_entropy_bwd",
    "msm_linear_cross_entropy_bwd_workspace_bytes",
]
SYMBOLS = list(__all__)


def declare(lib):
    """Argument types of the entry points of this module."""
    P, I64, F, SZ, E = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t, ctypes.c_int)
    lib.msm_embed_fwd.argtypes = [P, P, P, I64, I64, I64, F, E, E, P]
    lib.msm_embed_bwd.argtypes = [P, P, P, I64, I64, I64, F, E, E, P, SZ, P]
    lib.msm_embed_bwd_workspace_bytes.argtypes = [I64, I64, I64]
    lib.msm_block_norm_fwd.argtypes = [P] * 9 + [I64, I64, F, F, E, P]
    lib.msm_block_norm_bwd.argtypes = [P] * 14 + [I64, I64, F, E, P, SZ, P]
    lib.msm_block_norm_bwd_workspace_bytes.argtypes = [I64, I64, E]
    lib.msm_linear_cross_entropy_fwd.argtypes = [P] * 5 + [I64, I64, I64, F, E, P, SZ, P]
    lib.msm_linear_cross_entropy_bwd.argtypes = [P] * 8 + [I64, I64, I64, F, E, P, SZ, P]
    for which in ("fwd", "bwd"):
        getattr(lib, "msm_linear_cross_entropy_%s_workspace_bytes" % which).argtypes = [I64, I64, I64, E]
    for name in SYMBOLS:
        getattr(lib, name).restype = SZ if name.endswith("_workspace_bytes") else ctypes.c_int


from . import MsmError, _Owned, _workspace, load_library  # noqa: E402
from .ops import _check, _io_code, _ptr, _rows, _stream_handle  # noqa: E402


def msm_embed_fwd(ids, table, scale=1.0, *, io=None, y=None, stream=None):
    """scale * table[ids].  ids: (...) int64; table: (V, D) float32 or bfloat16.  Returns
    (..., D) in the dtype `io` (the table's by default); zeros where an id lies outside [0, V)."""
    import torch
    lib = load_library()
    own = _Owned(stream)
    dev = table.device
    if table.dim() != 2:
        raise ValueError("table has the shape (V, D)")
    V, D = table.shape
    io = (table.dtype if y is None else y.dtype) if io is None else io
    codes = _io_code(table.dtype), _io_code(io)
    shape = tuple(ids.shape)
    _check(ids, "ids", shape, torch.int64, dev)
    _check(table, "table", (V, D), table.dtype, dev)
    if y is None:
        y = own.empty(shape + (D,), io, dev)
    else:
        _check(y, "y", shape + (D,), io, dev)
    st = lib.msm_embed_fwd(_ptr(ids), _ptr(table), _ptr(y), ids.numel(), V, D, float(scale), *codes,
                           _stream_handle(stream, dev))
    own.done()
    if st != 0:
        raise MsmError(st, "msm_embed_fwd")
    return y


def msm_embed_bwd_workspace_bytes(tokens, V, D) -> int:
    return int(load_library().msm_embed_bwd_workspace_bytes(tokens, V, D))


def msm_embed_bwd(ids, dy, V, scale=1.0, *, table_dtype=None, dtable=None, workspace=None, stream=None):
    """Gradient of msm_embed_fwd's table.  ids: (...) int64; dy: (..., D).  Returns dtable (V, D)
    in `table_dtype` (dy's by default), every row written."""
    import torch
    lib = load_library()
    own = _Owned(stream)
    dev = dy.device
    shape = tuple(ids.shape)
    if dy.dim() != len(shape) + 1:
        raise ValueError("dy has the shape of ids and one dimension more")
    D = dy.shape[-1]
    table_dtype = (dy.dtype if dtable is None else dtable.dtype) if table_dtype is None else table_dtype
    codes = _io_code(table_dtype), _io_code(dy.dtype)
    _check(ids, "ids", shape, torch.int64, dev)
    _check(dy, "dy", shape + (D,), dy.dtype, dev)
    if dtable is None:
        dtable = own.empty((V, D), table_dtype, dev)
    else:
        _check(dtable, "dtable", (V, D), table_dtype, dev)
    tokens = ids.numel()
    ws, wsb = _workspace(int(lib.msm_embed_bwd_workspace_bytes(tokens, V, D)), workspace, dev, own)
    st = lib.msm_embed_bwd(_ptr(ids), _ptr(dy), _ptr(dtable), tokens, V, D, float(scale), *codes, _ptr(ws), wsb,
                           _stream_handle(stream, dev))
    own.done()
    if st != 0:
        raise MsmError(st, "msm_embed_bwd")
    return dtable


def _block_inputs(weight, o, post_weight, z, shape, io, dev):
    import torch
    D = shape[-1]
    if o is None and (post_weight is not None or z is not None):
        raise ValueError("post_weight and z belong to o")
    for t, nm in ((o, "o"), (z, "z")):
        if t is not None:
            _check(t, nm, shape, io, dev)
    for t, nm in ((weight, "weight"), (post_weight, "post_weight")):
        if t is not None:
            _check(t, nm, (D,), torch.float32, dev)


def msm_block_norm_fwd(r, weight=None, o=None, post_weight=None, z=None, scale=1.0, *, eps=1e-5, r_out=None, y=None,
                       rstd=None, post_rstd=None, return_stats=False, stream=None):
    """The norms after a block and before the next one, with the block's gate and residual scale:
    r_out = r + scale * post_weight * RMS(o) * silu(z), y = weight * RMS(r_out), over the last
    dimension.  r, o, z: (..., D) float32 or bfloat16; weight, post_weight: (D,) float32 or None
    (ones).  z None: no gate; o None: y = weight * RMS(r), and r_out is r.  r_out=r updates the
    stream in place.  Returns (r_out, y), or (r_out, y, rstd, post_rstd) with the (...) float32
    statistics that the backward takes when return_stats is true (post_rstd None without o)."""
    import torch
    lib = load_library()
    own = _Owned(stream)
    dev, io = r.device, r.dtype
    code = _io_code(io)
    if r.dim() == 0:
        raise ValueError("r has no dimension")
    rows, D = _rows(r)
    shape = tuple(r.shape)
    _check(r, "r", shape, io, dev)
    _block_inputs(weight, o, post_weight, z, shape, io, dev)
    # what the binding allocates needs no check
    if o is None:
        if post_rstd is not None or (r_out is not None and r_out is not r):
            raise ValueError("r_out and post_rstd belong to o")
        r_out = None
    elif r_out is None:
        r_out = own.empty(shape, io, dev)
    else:
        _check(r_out, "r_out", shape, io, dev)
    if y is None:
        y = own.empty(shape, io, dev)
    else:
        _check(y, "y", shape, io, dev)
    lead = shape[:-1]
    if rstd is not None:
        _check(rstd, "rstd", lead, torch.float32, dev)
    elif return_stats:
        rstd = own.empty(lead, torch.float32, dev)
    if post_rstd is not None:
        _check(post_rstd, "post_rstd", lead, torch.float32, dev)
    elif return_stats and o is not None:
        post_rstd = own.empty(lead, torch.float32, dev)
    st = lib.msm_block_norm_fwd(_ptr(r), _ptr(weight), _ptr(o), _ptr(post_weight), _ptr(z), _ptr(r_out), _ptr(y),
                                _ptr(rstd), _ptr(post_rstd), rows, D, float(scale), float(eps), code,
                                _stream_handle(stream, dev))
    own.done()
    if st != 0:
        raise MsmError(st, "msm_block_norm_fwd")
    r_out = r if r_out is None else r_out
    return (r_out, y, rstd, post_rstd) if return_stats else (r_out, y)


def msm_block_norm_bwd_workspace_bytes(rows, D, io) -> int:
    return int(load_library().msm_block_norm_bwd_workspace_bytes(rows, D, _io_code(io)))


def msm_block_norm_bwd(r_out, dy, rstd, weight=None, o=None, post_rstd=None, post_weight=None, z=None, scale=1.0, *,
                       dr_out=None, out=None, workspace=None, stream=None):
    """Gradients of sum(dy * y) + sum(dr_out * r_out) (dr_out None: zero) from the forward's r_out
    and statistics.  Returns a dict: dr, do (None without o), dz (None without z) in the I/O dtype,
    dweight and dpost_weight (D,) float32 (None where the weight is None)."""
    import torch
    lib = load_library()
    own = _Owned(stream)
    dev, io = r_out.device, r_out.dtype
    code = _io_code(io)
    if r_out.dim() == 0:
        raise ValueError("r_out has no dimension")
    rows, D = _rows(r_out)
    shape = tuple(r_out.shape)
    _check(r_out, "r_out", shape, io, dev)
    _check(dy, "dy", shape, io, dev)
    _check(rstd, "rstd", shape[:-1], torch.float32, dev)
    _block_inputs(weight, o, post_weight, z, shape, io, dev)
    if (o is None) != (post_rstd is None):
        raise ValueError("o and post_rstd are given together")
    if o is not None:
        _check(post_rstd, "post_rstd", shape[:-1], torch.float32, dev)
    if dr_out is not None:
        _check(dr_out, "dr_out", shape, io, dev)
    d = dict(out or {})
    for nm, wanted, shp, dt in (("dr", True, shape, io), ("do", o is not None, shape, io),
                                ("dz", z is not None, shape, io),
                                ("dweight", weight is not None, (D,), torch.float32),
                                ("dpost_weight", post_weight is not None, (D,), torch.float32)):
        if not wanted:
            d[nm] = None
            continue
        if nm not in d:
            d[nm] = own.empty(shp, dt, dev)
        else:
            _check(d[nm], nm, shp, dt, dev)
    ws, wsb = _workspace(int(lib.msm_block_norm_bwd_workspace_bytes(rows, D, code)), workspace, dev, own)
    st = lib.msm_block_norm_bwd(_ptr(r_out), _ptr(dy), _ptr(rstd), _ptr(weight), _ptr(o), _ptr(post_rstd),
                                _ptr(post_weight), _ptr(z), _ptr(dr_out), _ptr(d["dr"]), _ptr(d["do"]), _ptr(d["dz"]),
                                _ptr(d["dweight"]), _ptr(d["dpost_weight"]), rows, D, float(scale), code, _ptr(ws), wsb,
                                _stream_handle(stream, dev))
    own.done()
    if st != 0:
        raise MsmError(st, "msm_block_norm_bwd")
    return d


def msm_linear_cross_entropy_fwd_workspace_bytes(T, V, D, io) -> int:
    return int(load_library().msm_linear_cross_entropy_fwd_workspace_bytes(T, V, D, _io_code(io)))


def msm_linear_cross_entropy_bwd_workspace_bytes(T, V, D, io) -> int:
    return int(load_library().msm_linear_cross_entropy_bwd_workspace_bytes(T, V, D, _io_code(io)))


def _xent_sizes(x, weight, targets):
    import torch
    dev, io = x.device, x.dtype
    code = _io_code(io)
    if weight.dim() != 2:
        raise ValueError("weight has the shape (V, D)")
    V, D = weight.shape
    lead = tuple(targets.shape)
    _check(x, "x", lead + (D,), io, dev)
    _check(weight, "weight", (V, D), io, dev)
    _check(targets, "targets", lead, torch.int64, dev)
    return dev, io, code, lead, (targets.numel(), V, D)


def msm_linear_cross_entropy_fwd(x, weight, targets, scale=1.0, *, loss=None, lse=None, return_lse=False,
                                 workspace=None, stream=None):
    """Cross entropy of the logits scale * x @ weight.T, which are never in memory.  x: (..., D),
    weight: (V, D) float32 or bfloat16; targets: (...) int64.  Returns loss (...) float32, or
    (loss, lse) with the logarithms of the sums of exponentials, which the backward takes, when
    return_lse is true; both are 0 where a target lies outside [0, V)."""
    import torch
    lib = load_library()
    own = _Owned(stream)
    dev, io, code, lead, sizes = _xent_sizes(x, weight, targets)
    if loss is None:
        loss = own.empty(lead, torch.float32, dev)
    if return_lse and lse is None:
        lse = own.empty(lead, torch.float32, dev)
    for t, nm in ((loss, "loss"), (lse, "lse")):
        if t is not None:
            _check(t, nm, lead, torch.float32, dev)
    ws, wsb = _workspace(int(lib.msm_linear_cross_entropy_fwd_workspace_bytes(*sizes, code)), workspace, dev, own)
    st = lib.msm_linear_cross_entropy_fwd(_ptr(x), _ptr(weight), _ptr(targets), _ptr(loss), _ptr(lse), *sizes,
                                          float(scale), code, _ptr(ws), wsb, _stream_handle(stream, dev))
    own.done()
    if st != 0:
        raise MsmError(st, "msm_linear_cross_entropy_fwd")
    return (loss, lse) if return_lse else loss


def msm_linear_cross_entropy_bwd(x, weight, targets, lse, dloss, scale=1.0, *, dlse=None, weight_grad=True, out=None,
                                 workspace=None, stream=None):
    """Gradients of sum(dloss * loss) + sum(dlse * lse) (dlse None: zero) from the forward's lse.
    Returns a dict: dx (..., D) and dweight (V, D) in the I/O dtype (dweight None without
    weight_grad).  A row whose target lies outside [0, V) has dx = 0 and adds nothing to dweight."""
    import torch
    lib = load_library()
    own = _Owned(stream)
    dev, io, code, lead, sizes = _xent_sizes(x, weight, targets)
    for t, nm in ((lse, "lse"), (dloss, "dloss"), (dlse, "dlse")):
        if t is not None:
            _check(t, nm, lead, torch.float32, dev)
    d = dict(out or {})
    for nm, wanted, shp in (("dx", True, tuple(x.shape)), ("dweight", weight_grad, tuple(weight.shape))):
        if not wanted:
            d[nm] = None
            continue
        if nm not in d:
            d[nm] = own.empty(shp, io, dev)
        else:
            _check(d[nm], nm, shp, io, dev)
    ws, wsb = _workspace(int(lib.msm_linear_cross_entropy_bwd_workspace_bytes(*sizes, code)), workspace, dev, own)
    st = lib.msm_linear_cross_entropy_bwd(_ptr(x), _ptr(weight), _ptr(targets), _ptr(lse), _ptr(dloss), _ptr(dlse),
                                          _ptr(d["dx"]), _ptr(d["dweight"]), *sizes, float(scale), code, _ptr(ws), wsb,
                                          _stream_handle(stream, dev))
    own.done()
    if st != 0:
        raise MsmError(st, "msm_linear_cross_entropy_bwd")
    return d
