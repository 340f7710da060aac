"""ctypes binding of the local attention operators (include/rglru_attn.h).

Argument marshalling only, as in _abi.py: tensors become device pointers and
strides, outputs and workspaces are allocated through torch, a nonzero status
raises RGLRUError. A call runs on the device of its tensors, on `stream` or that
device's current stream, and allocates there; with a `stream` of its own the
caller orders it against the streams that made the inputs.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from ._abi import LIB, RGLRUError, _io_of, _ptr


class Strides(ctypes.Structure):
    """rglru_strides of include/rglru_attn.h."""
    _fields_ = [("batch", ctypes.c_longlong), ("token", ctypes.c_longlong),
                ("head", ctypes.c_longlong)]


def _declare(lib):
    vp, i32, sz, f32, f64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float,
                             ctypes.c_double)
    sp = ctypes.POINTER(Strides)
    lib.rglru_qk_norm_rope_fwd.restype = i32
    lib.rglru_qk_norm_rope_fwd.argtypes = ([vp, sp] * 2 + [vp] * 5 + [i32] * 6
                                           + [f64, f32, i32, vp])
    lib.rglru_qk_norm_rope_append.restype = i32
    lib.rglru_qk_norm_rope_append.argtypes = ([vp, sp] * 3 + [vp] * 7 + [i32] * 9
                                              + [f64, f32, i32, vp, vp])
    lib.rglru_qk_norm_rope_bwd_workspace_bytes.restype = sz
    lib.rglru_qk_norm_rope_bwd_workspace_bytes.argtypes = [i32] * 6
    lib.rglru_qk_norm_rope_bwd.restype = i32
    lib.rglru_qk_norm_rope_bwd.argtypes = ([vp, sp] * 2 + [vp] * 9 + [i32] * 6
                                           + [f64, f32, i32, vp, sz, vp])
    lib.rglru_local_attn_fwd.restype = i32
    lib.rglru_local_attn_fwd.argtypes = [vp, sp] * 3 + [vp] * 3 + [i32] * 8 + [f32, i32, vp, vp]
    lib.rglru_local_attn_bwd_workspace_bytes.restype = sz
    lib.rglru_local_attn_bwd_workspace_bytes.argtypes = [i32] * 9
    lib.rglru_local_attn_bwd.restype = i32
    lib.rglru_local_attn_bwd.argtypes = ([vp, sp] * 3 + [vp] * 7 + [i32] * 8
                                         + [f32, i32, vp, sz, vp, vp])
    lib.rglru_paged_attn_decode_workspace_bytes.restype = sz
    lib.rglru_paged_attn_decode_workspace_bytes.argtypes = [i32] * 9
    lib.rglru_paged_attn_decode.restype = i32
    lib.rglru_paged_attn_decode.argtypes = [vp] * 6 + [i32] * 9 + [f32, i32, vp, sz, vp, vp]


_declare(LIB)


@contextlib.contextmanager
def _on(dev, stream):
    """The call's device, and its stream as the one that allocations belong to."""
    with torch.cuda.device(dev):
        if stream is None:
            yield torch.cuda.current_stream(dev).cuda_stream
        else:
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def _heads(t, name, like=None):
    """(B, T, H, dh) of a tensor whose heads are contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dim() != 4:
        raise ValueError(f"{name} must be (B, T, heads, dh)")
    if like is not None and t.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return t.shape


def _view(t):
    """Pointer and strides of a (B, T, H, dh) tensor."""
    return t.data_ptr(), ctypes.byref(Strides(t.stride(0), t.stride(1), t.stride(2)))


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _shape(t, name, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _workspace(workspace, need, dev):
    if workspace is None:
        workspace = torch.empty(max(need, 256), device=dev, dtype=torch.uint8)
    return workspace


def _check(st, what):
    if st != 0:
        raise RGLRUError(st, what)


def rglru_qk_norm_rope_fwd(q, k, w_q=None, w_k=None, positions=None, *, rot=None, base=10000.0,
                           eps=1e-6, q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q (B, T, Hq, dh) and k (B, T, Hkv, dh), and the rotation of
    their first `rot` dims (all of them by default) by their positions (B, T; 0..T-1 by
    default), in one pass. q and k may be slices of a fused projection. Returns (q_out, k_out),
    dense."""
    B, T, Hq, dh = _heads(q, "q")
    Hkv = _heads(k, "k", q)[2]
    _shape(k, "k", (B, T, Hkv, dh))
    dt, dev = q.dtype, q.device
    io = _io_of(dt)
    _same_device(dev, k=k, w_q=w_q, w_k=w_k, positions=positions, q_out=q_out, k_out=k_out)
    with _on(dev, stream) as st:
        if q_out is None:
            q_out = torch.empty((B, T, Hq, dh), device=dev, dtype=dt)
        if k_out is None:
            k_out = torch.empty((B, T, Hkv, dh), device=dev, dtype=dt)
        _check(LIB.rglru_qk_norm_rope_fwd(
            *_view(q), *_view(k), _ptr(w_q, "w_q", dt, (dh,), optional=True),
            _ptr(w_k, "w_k", dt, (dh,), optional=True),
            _ptr(positions, "positions", torch.int32, (B, T), optional=True),
            _ptr(q_out, "q_out", dt, (B, T, Hq, dh)), _ptr(k_out, "k_out", dt, (B, T, Hkv, dh)),
            B, T, Hq, Hkv, dh, dh if rot is None else rot, base, eps, io, st),
            "rglru_qk_norm_rope_fwd")
    return q_out, k_out


def rglru_qk_norm_rope_append(q, k, v, k_cache, v_cache, page_table, positions, w_q=None,
                              w_k=None, *, rot=None, base=10000.0, eps=1e-6, q_out=None,
                              dev_status=None, stream=None):
    """The serving form: q normed and rotated into q_out (returned), k normed and rotated and v
    copied into their slots of the paged caches (pages, page_size, Hkv, dh), in place. Position
    p of row b lives in page page_table[b, p // page_size], slot p % page_size. Tokens at
    negative positions are padding; their rows of q_out are zeros when it is allocated here."""
    B, T, Hq, dh = _heads(q, "q")
    Hkv = _heads(k, "k", q)[2]
    _heads(v, "v", q)
    _shape(k, "k", (B, T, Hkv, dh))
    _shape(v, "v", (B, T, Hkv, dh))
    dt, dev = q.dtype, q.device
    io = _io_of(dt)
    _same_device(dev, k=k, v=v, k_cache=k_cache, v_cache=v_cache, page_table=page_table,
                 positions=positions, w_q=w_q, w_k=w_k, q_out=q_out, dev_status=dev_status)
    pages, page_size, max_pages = _cache_sizes(k_cache, v_cache, page_table, B, Hkv, dh)
    with _on(dev, stream) as st:
        if q_out is None:
            q_out = torch.zeros((B, T, Hq, dh), device=dev, dtype=dt)
        _check(LIB.rglru_qk_norm_rope_append(
            *_view(q), *_view(k), *_view(v), _ptr(w_q, "w_q", dt, (dh,), optional=True),
            _ptr(w_k, "w_k", dt, (dh,), optional=True),
            _ptr(positions, "positions", torch.int32, (B, T)),
            _ptr(q_out, "q_out", dt, (B, T, Hq, dh)), _ptr(k_cache, "k_cache", dt),
            _ptr(v_cache, "v_cache", dt), _ptr(page_table, "page_table", torch.int32), pages,
            page_size, max_pages, B, T, Hq, Hkv, dh, dh if rot is None else rot, base, eps, io,
            _ptr(dev_status, "dev_status", torch.int32, optional=True), st),
            "rglru_qk_norm_rope_append")
    return q_out


def _cache_sizes(k_cache, v_cache, page_table, B, Hkv, dh):
    if k_cache.dim() != 4 or page_table.dim() != 2:
        raise ValueError("a cache must be (pages, page_size, Hkv, dh) and page_table (B, max_pages)")
    pages, page_size = k_cache.shape[:2]
    _shape(k_cache, "k_cache", (pages, page_size, Hkv, dh))
    _shape(v_cache, "v_cache", (pages, page_size, Hkv, dh))
    _shape(page_table, "page_table", (B, page_table.shape[1]))
    return pages, page_size, page_table.shape[1]


def rglru_qk_norm_rope_bwd(q, k, dq_out, dk_out, w_q=None, w_k=None, positions=None, *, rot=None,
                           base=10000.0, eps=1e-6, workspace=None, out=None, stream=None):
    """Backward of rglru_qk_norm_rope_fwd. Returns a dict with dq, dk (dense, the I/O dtype) and
    dw_q, dw_k (fp32). `out` may hold preallocated outputs by name."""
    B, T, Hq, dh = _heads(q, "q")
    Hkv = _heads(k, "k", q)[2]
    _shape(k, "k", (B, T, Hkv, dh))
    dt, dev, f32 = q.dtype, q.device, torch.float32
    io = _io_of(dt)
    g = dict(out or {})
    _same_device(dev, k=k, dq_out=dq_out, dk_out=dk_out, w_q=w_q, w_k=w_k, positions=positions,
                 workspace=workspace, **g)
    with _on(dev, stream) as st:
        for name, shape, dtype in (("dq", (B, T, Hq, dh), dt), ("dk", (B, T, Hkv, dh), dt),
                                   ("dw_q", (dh,), f32), ("dw_k", (dh,), f32)):
            if g.get(name) is None:
                g[name] = torch.empty(shape, device=dev, dtype=dtype)
        need = LIB.rglru_qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hkv, dh, io)
        workspace = _workspace(workspace, need, dev)
        _check(LIB.rglru_qk_norm_rope_bwd(
            *_view(q), *_view(k), _ptr(w_q, "w_q", dt, (dh,), optional=True),
            _ptr(w_k, "w_k", dt, (dh,), optional=True),
            _ptr(positions, "positions", torch.int32, (B, T), optional=True),
            _ptr(dq_out, "dq_out", dt, (B, T, Hq, dh)),
            _ptr(dk_out, "dk_out", dt, (B, T, Hkv, dh)), _ptr(g["dq"], "dq", dt, (B, T, Hq, dh)),
            _ptr(g["dk"], "dk", dt, (B, T, Hkv, dh)), _ptr(g["dw_q"], "dw_q", f32, (dh,)),
            _ptr(g["dw_k"], "dw_k", f32, (dh,)), B, T, Hq, Hkv, dh, dh if rot is None else rot,
            base, eps, io, _ptr(workspace, "workspace"),
            workspace.numel() * workspace.element_size(), st), "rglru_qk_norm_rope_bwd")
    return g


def rglru_local_attn_fwd(q, k, v, *, window=0, sinks=0, scale=None, lens=None, out=None, lse=None,
                         want_lse=True, dev_status=None, stream=None):
    """Attention of q (B, T, Hq, dh) over k, v (B, S, Hkv, dh): causal, the last `window` keys
    (0: all) and the first `sinks` keys; query t stands at position t + S - T. `scale` is
    1 / sqrt(dh) by default. With `lens` (B, int32; S == T) row b has lens[b] tokens, and rows
    past them are left as they were in given outputs, zeros (and -inf in lse) in ones allocated
    here. Returns (out, lse), lse (B, Hq, T) or None when it is neither wanted nor given."""
    B, T, Hq, dh = _heads(q, "q")
    _, S, Hkv, _ = _heads(k, "k", q)
    _heads(v, "v", q)
    _shape(k, "k", (B, S, Hkv, dh))
    _shape(v, "v", (B, S, Hkv, dh))
    dt, dev = q.dtype, q.device
    io = _io_of(dt)
    _same_device(dev, k=k, v=v, lens=lens, out=out, lse=lse, dev_status=dev_status)
    with _on(dev, stream) as st:
        if out is None:
            make = torch.empty if lens is None else torch.zeros
            out = make((B, T, Hq, dh), device=dev, dtype=dt)
        if lse is None and want_lse:
            lse = torch.empty((B, Hq, T), device=dev, dtype=torch.float32)
            if lens is not None:
                lse.fill_(float("-inf"))
        _check(LIB.rglru_local_attn_fwd(
            *_view(q), *_view(k), *_view(v), _ptr(lens, "lens", torch.int32, (B,), optional=True),
            _ptr(out, "out", dt, (B, T, Hq, dh)),
            _ptr(lse, "lse", torch.float32, (B, Hq, T), optional=True), B, T, S, Hq, Hkv, dh,
            window, sinks, dh ** -0.5 if scale is None else scale, io,
            _ptr(dev_status, "dev_status", torch.int32, optional=True), st),
            "rglru_local_attn_fwd")
    return out, lse


def rglru_local_attn_bwd(q, k, v, out, lse, dout, *, window=0, sinks=0, scale=None, lens=None,
                         workspace=None, grads=None, dev_status=None, stream=None):
    """Backward of rglru_local_attn_fwd from its inputs, its out and lse, and dout. Returns a
    dict with dq, dk, dv (dense, the I/O dtype). `grads` may hold preallocated outputs by name;
    with `lens`, rows past a sequence are left as they were there, zeros otherwise."""
    B, T, Hq, dh = _heads(q, "q")
    _, S, Hkv, _ = _heads(k, "k", q)
    _heads(v, "v", q)
    _shape(k, "k", (B, S, Hkv, dh))
    _shape(v, "v", (B, S, Hkv, dh))
    dt, dev = q.dtype, q.device
    io = _io_of(dt)
    g = dict(grads or {})
    _same_device(dev, k=k, v=v, out=out, lse=lse, dout=dout, lens=lens, workspace=workspace,
                 dev_status=dev_status, **g)
    with _on(dev, stream) as st:
        make = torch.empty if lens is None else torch.zeros
        for name, shape in (("dq", (B, T, Hq, dh)), ("dk", (B, S, Hkv, dh)),
                            ("dv", (B, S, Hkv, dh))):
            if g.get(name) is None:
                g[name] = make(shape, device=dev, dtype=dt)
        need = LIB.rglru_local_attn_bwd_workspace_bytes(B, T, S, Hq, Hkv, dh, window, sinks, io)
        workspace = _workspace(workspace, need, dev)
        _check(LIB.rglru_local_attn_bwd(
            *_view(q), *_view(k), *_view(v), _ptr(out, "out", dt, (B, T, Hq, dh)),
            _ptr(lse, "lse", torch.float32, (B, Hq, T)), _ptr(dout, "dout", dt, (B, T, Hq, dh)),
            _ptr(lens, "lens", torch.int32, (B,), optional=True),
            _ptr(g["dq"], "dq", dt, (B, T, Hq, dh)), _ptr(g["dk"], "dk", dt, (B, S, Hkv, dh)),
            _ptr(g["dv"], "dv", dt, (B, S, Hkv, dh)), B, T, S, Hq, Hkv, dh, window, sinks,
            dh ** -0.5 if scale is None else scale, io, _ptr(workspace, "workspace"),
            workspace.numel() * workspace.element_size(),
            _ptr(dev_status, "dev_status", torch.int32, optional=True), st),
            "rglru_local_attn_bwd")
    return g


def rglru_paged_attn_decode(q, k_cache, v_cache, page_table, lens, *, window=0, sinks=0,
                            scale=None, out=None, workspace=None, dev_status=None, stream=None):
    """Attention of one new token of each sequence, q (B, Hq, dh), over its paged cache (pages,
    page_size, Hkv, dh): its last `window` keys (0: all) and its first `sinks`, of lens[b] keys
    (the new token's own among them; 0: the row of out is zeros). Returns out (B, Hq, dh)."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError("q must be a CUDA tensor (the library has no CPU path)")
    if q.dim() != 3:
        raise ValueError("q must be (B, Hq, dh)")
    B, Hq, dh = q.shape
    dt, dev = q.dtype, q.device
    io = _io_of(dt)
    _same_device(dev, k_cache=k_cache, v_cache=v_cache, page_table=page_table, lens=lens, out=out,
                 workspace=workspace, dev_status=dev_status)
    if k_cache.dim() != 4:
        raise ValueError("a cache must be (pages, page_size, Hkv, dh)")
    Hkv = k_cache.shape[2]
    pages, page_size, max_pages = _cache_sizes(k_cache, v_cache, page_table, B, Hkv, dh)
    with _on(dev, stream) as st:
        if out is None:
            out = torch.empty((B, Hq, dh), device=dev, dtype=dt)
        need = LIB.rglru_paged_attn_decode_workspace_bytes(B, Hq, Hkv, dh, page_size, max_pages,
                                                           window, sinks, io)
        workspace = _workspace(workspace, need, dev)
        _check(LIB.rglru_paged_attn_decode(
            _ptr(q, "q", dt, (B, Hq, dh)), _ptr(k_cache, "k_cache", dt),
            _ptr(v_cache, "v_cache", dt), _ptr(page_table, "page_table", torch.int32),
            _ptr(lens, "lens", torch.int32, (B,)), _ptr(out, "out", dt, (B, Hq, dh)), pages,
            page_size, max_pages, B, Hq, Hkv, dh, window, sinks,
            dh ** -0.5 if scale is None else scale, io, _ptr(workspace, "workspace"),
            workspace.numel() * workspace.element_size(),
            _ptr(dev_status, "dev_status", torch.int32, optional=True), st),
            "rglru_paged_attn_decode")
    return out
