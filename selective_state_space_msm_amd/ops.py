"""Python binding of the block operators of libmsm.so: the gated delta rule, layer norm, and the
norm and clipping of gradients.  Same manner as the scan's binding: names of the C entry points,
argument checks and marshalling only, every step in the library's HIP kernels.

    o, S = msm_delta_rule_fwd(q, k, v, g, beta, return_last_state=True)       # chunked prefill
    grads = msm_delta_rule_bwd(q, k, v, g, beta, do)                          # training
    o = msm_delta_rule_step(q, k, v, g, beta, S)                              # one token, S in place
    y, mean, rstd = msm_layer_norm_fwd(x, weight, bias, return_stats=True)
    grads = msm_layer_norm_bwd(x, dy, mean, rstd, weight, bias_grad=True)
    norm = msm_grad_clip(list_of_gradients, max_norm)                         # in place
"""
from __future__ import annotations

import ctypes
from array import array

__all__ = [
    "msm_delta_rule_fwd_workspace_bytes", "msm_delta_rule_bwd_workspace_bytes",
    "msm_delta_rule_fwd", "msm_delta_rule_bwd", "msm_delta_rule_step", "msm_layer_norm_fwd",
    "msm_layer_norm_bwd", "msm_layer_norm_bwd_workspace_bytes", "msm_grad_norm", "msm_grad_clip",
    "msm_grad_norm_workspace_bytes",
]
SYMBOLS = list(__all__)


def declare(lib):
    """Argument types of the entry points of this module."""
    P, I64, F, I32, SZ, E = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int32,
                             ctypes.c_size_t, ctypes.c_int)
    for name in ("msm_delta_rule_fwd_workspace_bytes", "msm_delta_rule_bwd_workspace_bytes"):
        fn = getattr(lib, name)
        fn.argtypes = [I64] * 6 + [I32, E]
        fn.restype = SZ
    lib.msm_delta_rule_fwd.argtypes = [P] * 9 + [I64] * 6 + [F, E, P, SZ, P]
    lib.msm_delta_rule_bwd.argtypes = [P] * 15 + [I64] * 6 + [F, E, P, SZ, P]
    lib.msm_delta_rule_step.argtypes = [P] * 7 + [I64] * 5 + [F, E, P]
    lib.msm_layer_norm_fwd.argtypes = [P] * 6 + [I64, I64, F, E, P]
    lib.msm_layer_norm_bwd_workspace_bytes.argtypes = [I64, I64, E]
    lib.msm_layer_norm_bwd_workspace_bytes.restype = SZ
    lib.msm_layer_norm_bwd.argtypes = [P] * 8 + [I64, I64, E, P, SZ, P]
    lib.msm_grad_norm_workspace_bytes.argtypes = [I64]
    lib.msm_grad_norm_workspace_bytes.restype = SZ
    lib.msm_grad_norm.argtypes = [P, P, P, I64, P, P, SZ, P]
    lib.msm_grad_clip.argtypes = [P, P, P, P, I64, F, F, P, P, SZ, P]
    for name in ("msm_delta_rule_fwd", "msm_delta_rule_bwd", "msm_delta_rule_step",
                 "msm_layer_norm_fwd", "msm_layer_norm_bwd", "msm_grad_norm", "msm_grad_clip"):
        getattr(lib, name).restype = ctypes.c_int


from . import MsmError, _on_gpu, _Owned, _workspace, load_library  # noqa: E402
from . import _check as _explain  # noqa: E402
from . import _io_code as _code  # noqa: E402


# A small call's time is the time to make it: the checks below cost one comparison each while they
# hold, addresses go to ctypes as plain numbers, and the current stream is asked for its handle
# without an object around it.

def _check(t, name, shape, dtype, device):
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        _explain(t, name, shape, dtype, device)


def _io_code(io):
    import torch
    if io is torch.bfloat16:
        return 1
    return 0 if io is torch.float32 else _code(io)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_handle(stream, device):
    import torch
    _on_gpu(stream, device)
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


def msm_delta_rule_fwd_workspace_bytes(Bt, L, Hk, H, K, V, io, packed=False) -> int:
    return int(load_library().msm_delta_rule_fwd_workspace_bytes(Bt, L, Hk, H, K, V,
                                                                 int(bool(packed)), _io_code(io)))


def msm_delta_rule_bwd_workspace_bytes(Bt, L, Hk, H, K, V, io, packed=False) -> int:
    return int(load_library().msm_delta_rule_bwd_workspace_bytes(Bt, L, Hk, H, K, V,
                                                                 int(bool(packed)), _io_code(io)))


def _delta_sizes(q, k, v, g, beta, seq_offsets):
    import torch
    dev, io = q.device, q.dtype
    _io_code(io)
    if seq_offsets is None:
        if q.dim() != 4 or v.dim() != 4:
            raise ValueError("q, k, v have the shapes (Bt, L, heads, size)")
        lead = tuple(q.shape[:2])
        Bt, L = lead
    else:
        if q.dim() != 3 or v.dim() != 3:
            raise ValueError("packed q, k, v have the shapes (tokens, heads, size)")
        if seq_offsets.dim() != 1 or seq_offsets.numel() < 2:
            raise ValueError("seq_offsets has the shape (sequences + 1,)")
        lead = tuple(q.shape[:1])
        Bt, L = seq_offsets.numel() - 1, lead[0]
        _check(seq_offsets, "seq_offsets", (Bt + 1,), torch.int32, dev)
    Hk, K = q.shape[-2:]
    H, V = v.shape[-2:]
    _check(q, "q", lead + (Hk, K), io, dev)
    _check(k, "k", lead + (Hk, K), io, dev)
    _check(v, "v", lead + (H, V), io, dev)
    _check(g, "g", lead + (H,), torch.float32, dev)
    _check(beta, "beta", lead + (H,), torch.float32, dev)
    return dev, lead, (Bt, L, Hk, H, K, V), _io_code(io)


def msm_delta_rule_fwd(q, k, v, g, beta, scale=None, *, S0=None, seq_offsets=None, o=None,
                       last_S=None, return_last_state=False, workspace=None, stream=None):
    """Gated delta rule over whole sequences.  q, k: (Bt, L, Hk, K); v: (Bt, L, H, V) in float32
    or bfloat16; g (log decay), beta: (Bt, L, H) float32; S0: optional (Bt, H, K, V) float32.
    With seq_offsets (int32, sequences + 1) the token arrays are packed, (tokens, heads, size).
    scale defaults to K ** -0.5.  Returns o, or (o, last_S) when return_last_state is true."""
    import torch
    lib = load_library()
    own = _Owned(stream)
    dev, lead, sizes, io = _delta_sizes(q, k, v, g, beta, seq_offsets)
    Bt, L, Hk, H, K, V = sizes
    if o is None:
        o = own.empty(lead + (H, V), v.dtype, dev)
    _check(o, "o", lead + (H, V), v.dtype, dev)
    if return_last_state and last_S is None:
        last_S = own.empty((Bt, H, K, V), torch.float32, dev)
    for t, nm in ((S0, "S0"), (last_S, "last_S")):
        if t is not None:
            _check(t, nm, (Bt, H, K, V), torch.float32, dev)
    nbytes = int(lib.msm_delta_rule_fwd_workspace_bytes(*sizes, int(seq_offsets is not None), io))
    ws, wsb = _workspace(nbytes, workspace, dev, own)
    st = lib.msm_delta_rule_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(seq_offsets),
                                _ptr(S0), _ptr(o), _ptr(last_S), *sizes,
                                float(K ** -0.5 if scale is None else scale), io, _ptr(ws), wsb,
                                _stream_handle(stream, dev))
    own.done()
    if st != 0:
        raise MsmError(st, "msm_delta_rule_fwd")
    return (o, last_S) if return_last_state else o


def msm_delta_rule_bwd(q, k, v, g, beta, do, scale=None, *, S0=None, dlast_S=None,
                       seq_offsets=None, state_grads=False, out=None, workspace=None, stream=None):
    """Gradients of sum(do * o) + <dlast_S, last_S>.  Returns a dict: dq, dk, dv in the I/O dtype,
    dg, dbeta float32 and, with state_grads, dS0 (Bt, H, K, V) float32.  Arguments as
    msm_delta_rule_fwd; the forward is recomputed inside."""
    import torch
    lib = load_library()
    own = _Owned(stream)
    dev, lead, sizes, io = _delta_sizes(q, k, v, g, beta, seq_offsets)
    Bt, L, Hk, H, K, V = sizes
    _check(do, "do", lead + (H, V), v.dtype, dev)
    for t, nm in ((S0, "S0"), (dlast_S, "dlast_S")):
        if t is not None:
            _check(t, nm, (Bt, H, K, V), torch.float32, dev)
    d = dict(out or {})
    grads = [("dq", lead + (Hk, K), v.dtype), ("dk", lead + (Hk, K), v.dtype),
             ("dv", lead + (H, V), v.dtype), ("dg", lead + (H,), torch.float32),
             ("dbeta", lead + (H,), torch.float32)]
    if state_grads or "dS0" in d:
        grads.append(("dS0", (Bt, H, K, V), torch.float32))
    for nm, shp, dt in grads:
        if nm not in d:
            d[nm] = own.empty(shp, dt, dev)
        _check(d[nm], nm, shp, dt, dev)
    nbytes = int(lib.msm_delta_rule_bwd_workspace_bytes(*sizes, int(seq_offsets is not None), io))
    ws, wsb = _workspace(nbytes, workspace, dev, own)
    st = lib.msm_delta_rule_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(seq_offsets),
                                _ptr(S0), _ptr(do), _ptr(dlast_S), _ptr(d["dq"]), _ptr(d["dk"]),
                                _ptr(d["dv"]), _ptr(d["dg"]), _ptr(d["dbeta"]), _ptr(d.get("dS0")),
                                *sizes, float(K ** -0.5 if scale is None else scale), io, _ptr(ws),
                                wsb, _stream_handle(stream, dev))
    own.done()
    if st != 0:
        raise MsmError(st, "msm_delta_rule_bwd")
    return d


def msm_delta_rule_step(q, k, v, g, beta, S, scale=None, *, o=None, stream=None):
    """One token: q, k (Bt, Hk, K), v (Bt, H, V) in the I/O dtype; g, beta (Bt, H) float32; the
    states S (Bt, H, K, V) float32 are updated in place.  Returns o (Bt, H, V)."""
    import torch
    lib = load_library()
    own = _Owned(stream)
    dev, io = q.device, _io_code(q.dtype)
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v have the shapes (Bt, heads, size)")
    Bt, Hk, K = q.shape
    H, V = v.shape[-2:]
    _check(q, "q", (Bt, Hk, K), q.dtype, dev)
    _check(k, "k", (Bt, Hk, K), q.dtype, dev)
    _check(v, "v", (Bt, H, V), q.dtype, dev)
    _check(g, "g", (Bt, H), torch.float32, dev)
    _check(beta, "beta", (Bt, H), torch.float32, dev)
    _check(S, "S", (Bt, H, K, V), torch.float32, dev)
    if o is None:
        o = own.empty((Bt, H, V), v.dtype, dev)
    _check(o, "o", (Bt, H, V), v.dtype, dev)
    st = lib.msm_delta_rule_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S), _ptr(o),
                                 Bt, Hk, H, K, V, float(K ** -0.5 if scale is None else scale), io,
                                 _stream_handle(stream, dev))
    own.done()
    if st != 0:
        raise MsmError(st, "msm_delta_rule_step")
    return o


def msm_layer_norm_bwd_workspace_bytes(rows, D, io) -> int:
    return int(load_library().msm_layer_norm_bwd_workspace_bytes(rows, D, _io_code(io)))


def _rows(x):
    D = x.shape[-1] if x.dim() else 0
    return (x.numel() // D if D else 0), D


def msm_layer_norm_fwd(x, weight=None, bias=None, *, eps=1e-5, y=None, mean=None, rstd=None,
                       return_stats=False, stream=None):
    """Layer norm over the last dimension.  x: (..., D) float32 or bfloat16; weight, bias: (D,)
    float32 or None.  Returns y, or (y, mean, rstd) with the (...) float32 statistics that the
    backward takes when return_stats is true."""
    import torch
    lib = load_library()
    own = _Owned(stream)
    dev, io = x.device, _io_code(x.dtype)
    rows, D = _rows(x)
    lead = tuple(x.shape[:-1])
    _check(x, "x", tuple(x.shape), x.dtype, dev)
    for t, nm in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _check(t, nm, (D,), torch.float32, dev)
    if y is None:
        y = own.empty(tuple(x.shape), x.dtype, dev)
    _check(y, "y", tuple(x.shape), x.dtype, dev)
    if return_stats:
        mean = own.empty(lead, torch.float32, dev) if mean is None else mean
        rstd = own.empty(lead, torch.float32, dev) if rstd is None else rstd
    for t, nm in ((mean, "mean"), (rstd, "rstd")):
        if t is not None:
            _check(t, nm, lead, torch.float32, dev)
    st = lib.msm_layer_norm_fwd(_ptr(x), _ptr(weight), _ptr(bias), _ptr(y), _ptr(mean), _ptr(rstd),
                                rows, D, float(eps), io, _stream_handle(stream, dev))
    own.done()
    if st != 0:
        raise MsmError(st, "msm_layer_norm_fwd")
    return (y, mean, rstd) if return_stats else y


def msm_layer_norm_bwd(x, dy, mean, rstd, weight=None, *, bias_grad=False, out=None,
                       workspace=None, stream=None):
    """Gradients of sum(dy * y) from the forward's statistics.  Returns a dict: dx in the I/O
    dtype, dweight (D,) float32 (None without weight) and dbias (D,) float32 (None without
    bias_grad)."""
    import torch
    lib = load_library()
    own = _Owned(stream)
    dev, io = x.device, _io_code(x.dtype)
    rows, D = _rows(x)
    lead = tuple(x.shape[:-1])
    _check(x, "x", tuple(x.shape), x.dtype, dev)
    _check(dy, "dy", tuple(x.shape), x.dtype, dev)
    _check(mean, "mean", lead, torch.float32, dev)
    _check(rstd, "rstd", lead, torch.float32, dev)
    if weight is not None:
        _check(weight, "weight", (D,), torch.float32, dev)
    d = dict(out or {})
    for nm, wanted, shp, dt in (("dx", True, tuple(x.shape), x.dtype),
                                ("dweight", weight is not None, (D,), torch.float32),
                                ("dbias", bias_grad, (D,), torch.float32)):
        if not wanted:
            d[nm] = None
            continue
        if nm not in d:
            d[nm] = own.empty(shp, dt, dev)
        _check(d[nm], nm, shp, dt, dev)
    nbytes = 0
    if d["dweight"] is not None or d["dbias"] is not None:
        nbytes = int(lib.msm_layer_norm_bwd_workspace_bytes(rows, D, io))
    ws, wsb = _workspace(nbytes, workspace, dev, own)
    st = lib.msm_layer_norm_bwd(_ptr(x), _ptr(weight), _ptr(dy), _ptr(mean), _ptr(rstd),
                                _ptr(d["dx"]), _ptr(d["dweight"]), _ptr(d["dbias"]), rows, D, io,
                                _ptr(ws), wsb, _stream_handle(stream, dev))
    own.done()
    if st != 0:
        raise MsmError(st, "msm_layer_norm_bwd")
    return d


def msm_grad_norm_workspace_bytes(count) -> int:
    return int(load_library().msm_grad_norm_workspace_bytes(count))


def _tensor_list(tensors, what):
    """Host arrays of addresses, element counts and dtypes of a list of contiguous tensors on one
    device."""
    import torch
    T = torch.Tensor
    index = set(map(T.get_device, tensors))
    if len(index) != 1:
        raise ValueError("%s are on several devices" % what)
    if not all(map(T.is_contiguous, tensors)):
        i = [t.is_contiguous() for t in tensors].index(False)
        raise ValueError("%s[%d] must be contiguous" % (what, i))
    code = {torch.float32: 0, torch.bfloat16: 1}
    try:
        types = [code[t.dtype] for t in tensors]
    except KeyError as e:
        raise ValueError("unsupported dtype %s in %s" % (e.args[0], what)) from None
    return (array("Q", map(T.data_ptr, tensors)), array("q", map(T.numel, tensors)), array("i", types))


def _address(a):
    return None if a is None else a.buffer_info()[0]


def msm_grad_norm(grads, *, workspace=None, stream=None):
    """2-norm over all tensors of a list (float32 and bfloat16 mixed freely), as a float32 tensor
    without dimensions on their device."""
    import torch
    lib = load_library()
    own = _Owned(stream)
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    ptrs, numel, types = _tensor_list(grads, "grads")
    dev = grads[0].device
    norm = own.empty((), torch.float32, dev)
    ws, wsb = _workspace(int(lib.msm_grad_norm_workspace_bytes(len(grads))), workspace, dev, own)
    st = lib.msm_grad_norm(_address(ptrs), _address(numel), _address(types), len(grads), _ptr(norm),
                           _ptr(ws), wsb, _stream_handle(stream, dev))
    own.done()
    if st != 0:
        raise MsmError(st, "msm_grad_norm")
    return norm


def msm_grad_clip(grads, max_norm, *, eps=1e-6, out=None, workspace=None, stream=None):
    """Scales a list of gradients by min(1, max_norm / (norm + eps)), in place or into the tensors
    of `out`.  What is written must not overlap anything else: in place, no tensor is listed twice.
    Returns the norm before clipping, a float32 tensor without dimensions."""
    import torch
    lib = load_library()
    own = _Owned(stream)
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    ptrs, numel, types = _tensor_list(grads, "grads")
    dev = grads[0].device
    optrs = None
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError("out has %d tensors, expected %d" % (len(out), len(grads)))
        optrs, onumel, otypes = _tensor_list(out, "out")
        if onumel != numel or otypes != types:
            raise ValueError("a tensor of out differs from its gradient in size or dtype")
        if out[0].device != dev:
            raise ValueError("out is on %s, expected %s" % (out[0].device, dev))
    norm = own.empty((), torch.float32, dev)
    ws, wsb = _workspace(int(lib.msm_grad_norm_workspace_bytes(len(grads))), workspace, dev, own)
    st = lib.msm_grad_clip(_address(ptrs), _address(optrs), _address(numel), _address(types),
                           len(grads), float(max_norm), float(eps), _ptr(norm), _ptr(ws), wsb,
                           _stream_handle(stream, dev))
    own.done()
    if st != 0:
        raise MsmError(st, "msm_grad_clip")
    return norm
