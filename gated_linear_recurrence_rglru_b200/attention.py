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

from ._abi import LIB, RGLRUError, _io_of


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


# The handle of a device's current stream; through the Stream object that torch builds
# for it, a call would spend 3 us more on the host.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _on:
    """The call's device, and its stream as the one that allocations belong to; gives the
    stream's handle. Nothing is switched when both are current already."""
    __slots__ = ("index", "stream", "held")

    def __init__(self, index, stream):
        self.index, self.stream, self.held = index, stream, None

    def __enter__(self):
        if self.stream is None and torch.cuda.current_device() == self.index:
            return _current_stream(self.index)
        self.held = contextlib.ExitStack()
        self.held.enter_context(torch.cuda.device(self.index))
        if self.stream is None:
            return _current_stream(self.index)
        self.held.enter_context(torch.cuda.stream(self.stream))
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.held is not None:
            self.held.close()


def _place(t, name, index):
    """Refuses what is not a tensor on the call's device (index None: any CUDA device)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _p(t, name, dtype, shape, index, optional=False):
    """Pointer of a dense tensor on the call's device; dtype or shape None: not looked at."""
    try:        # the checks below in one expression: what a good call pays for
        if (t.get_device() == index and (shape is None or t.shape == shape) and t.dtype is dtype
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    _place(t, name, index)
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _view(t, name, dtype, shape, index):
    """Pointer and strides (None: dense) of a (B, T, H, dh) tensor whose heads are contiguous;
    dtype, shape or index None: any."""
    _place(t, name, index)
    if t.dim() != 4:
        raise ValueError(f"{name} must be (B, T, heads, dh)")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), None
    sb, st, sh, sd = t.stride()
    if sd != 1 and t.shape[3] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return t.data_ptr(), Strides(sb, st, sh)


def _workspace(workspace, need, dev):
    if workspace is None:
        workspace = torch.empty(max(need, 256), device=dev, dtype=torch.uint8)
    return workspace


def _check(st, what):
    if st != 0:
        raise RGLRUError(st, what)


def _sizes(q, k, v=None):
    """What the shapes of q (B, T, Hq, dh) and k, v (B, S, Hkv, dh) say, and their views."""
    qv = _view(q, "q", None, None, None)
    index, dt = q.get_device(), q.dtype
    io = _io_of(dt)
    B, T, Hq, dh = q.shape
    kv = _view(k, "k", dt, None, index)
    _, S, Hkv, _ = k.shape
    if k.shape != (B, S, Hkv, dh):
        raise ValueError(f"k must have shape {(B, S, Hkv, dh)}, got {tuple(k.shape)}")
    views = (*qv, *kv)
    if v is not None:
        views += _view(v, "v", dt, (B, S, Hkv, dh), index)
    return views, index, dt, io, B, T, S, Hq, Hkv, dh


def _same_length(S, T):
    if S != T:
        raise ValueError(f"k must have q's {T} tokens, got {S}")


def rglru_qk_norm_rope_fwd(q, k, w_q=None, w_k=None, positions=None, *, rot=None, base=10000.0,
                           eps=1e-6, q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q (B, T, Hq, dh) and k (B, T, Hkv, dh), and the rotation of
    their first `rot` dims (all of them by default) by their positions (B, T; 0..T-1 by
    default), in one pass. q and k may be slices of a fused projection. Returns (q_out, k_out),
    dense."""
    views, dev, dt, io, B, T, S, Hq, Hkv, dh = _sizes(q, k)
    _same_length(S, T)
    with _on(dev, stream) as st:
        if q_out is None:
            q_out = q.new_empty((B, T, Hq, dh))
        if k_out is None:
            k_out = q.new_empty((B, T, Hkv, dh))
        _check(LIB.rglru_qk_norm_rope_fwd(
            *views, _p(w_q, "w_q", dt, (dh,), dev, True), _p(w_k, "w_k", dt, (dh,), dev, True),
            _p(positions, "positions", torch.int32, (B, T), dev, True),
            _p(q_out, "q_out", dt, (B, T, Hq, dh), dev), _p(k_out, "k_out", dt, (B, T, Hkv, dh), dev),
            B, T, Hq, Hkv, dh, dh if rot is None else rot, base, eps, io, st),
            "rglru_qk_norm_rope_fwd")
    return q_out, k_out


def _cache(k_cache, v_cache, page_table, dt, B, Hkv, dh, dev):
    """Pointers and sizes of the caches and the page table."""
    kc = _p(k_cache, "k_cache", dt, None, dev)
    if k_cache.dim() != 4:
        raise ValueError("a cache must be (pages, page_size, Hkv, dh)")
    pages, page_size = k_cache.shape[:2]
    if k_cache.shape != (pages, page_size, Hkv, dh):
        raise ValueError(f"k_cache must have shape {(pages, page_size, Hkv, dh)}, "
                         f"got {tuple(k_cache.shape)}")
    vc = _p(v_cache, "v_cache", dt, k_cache.shape, dev)
    table = _p(page_table, "page_table", torch.int32, None, dev)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table must have shape ({B}, max_pages), got {tuple(page_table.shape)}")
    return kc, vc, table, pages, page_size, page_table.shape[1]


def rglru_qk_norm_rope_append(q, k, v, k_cache, v_cache, page_table, positions, w_q=None,
                              w_k=None, *, rot=None, base=10000.0, eps=1e-6, q_out=None,
                              dev_status=None, stream=None):
    """The serving form: q normed and rotated into q_out (returned), k normed and rotated and v
    copied into their slots of the paged caches (pages, page_size, Hkv, dh), in place. Position
    p of row b lives in page page_table[b, p // page_size], slot p % page_size. Tokens at
    negative positions are padding: their rows of q_out are zeros and no slot is written."""
    views, dev, dt, io, B, T, S, Hq, Hkv, dh = _sizes(q, k, v)
    _same_length(S, T)
    kc, vc, table, pages, page_size, max_pages = _cache(k_cache, v_cache, page_table, dt, B, Hkv,
                                                        dh, dev)
    with _on(dev, stream) as st:
        if q_out is None:
            q_out = q.new_empty((B, T, Hq, dh))
        _check(LIB.rglru_qk_norm_rope_append(
            *views, _p(w_q, "w_q", dt, (dh,), dev, True), _p(w_k, "w_k", dt, (dh,), dev, True),
            _p(positions, "positions", torch.int32, (B, T), dev),
            _p(q_out, "q_out", dt, (B, T, Hq, dh), dev), kc, vc, table, pages, page_size,
            max_pages, B, T, Hq, Hkv, dh, dh if rot is None else rot, base, eps, io,
            _p(dev_status, "dev_status", torch.int32, None, dev, True), st),
            "rglru_qk_norm_rope_append")
    return q_out


def rglru_qk_norm_rope_bwd(q, k, dq_out, dk_out, w_q=None, w_k=None, positions=None, *, rot=None,
                           base=10000.0, eps=1e-6, workspace=None, out=None, stream=None):
    """Backward of rglru_qk_norm_rope_fwd. Returns a dict with dq, dk (dense, the I/O dtype) and
    dw_q, dw_k (fp32). `out` may hold preallocated outputs by name."""
    views, dev, dt, io, B, T, S, Hq, Hkv, dh = _sizes(q, k)
    _same_length(S, T)
    g, f32 = dict(out or {}), torch.float32
    with _on(dev, stream) as st:
        for name, shape, dtype in (("dq", (B, T, Hq, dh), dt), ("dk", (B, T, Hkv, dh), dt),
                                   ("dw_q", (dh,), f32), ("dw_k", (dh,), f32)):
            if g.get(name) is None:
                g[name] = torch.empty(shape, device=q.device, dtype=dtype)
        need = LIB.rglru_qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hkv, dh, io)
        workspace = _workspace(workspace, need, q.device)
        _check(LIB.rglru_qk_norm_rope_bwd(
            *views, _p(w_q, "w_q", dt, (dh,), dev, True), _p(w_k, "w_k", dt, (dh,), dev, True),
            _p(positions, "positions", torch.int32, (B, T), dev, True),
            _p(dq_out, "dq_out", dt, (B, T, Hq, dh), dev),
            _p(dk_out, "dk_out", dt, (B, T, Hkv, dh), dev),
            _p(g["dq"], "dq", dt, (B, T, Hq, dh), dev), _p(g["dk"], "dk", dt, (B, T, Hkv, dh), dev),
            _p(g["dw_q"], "dw_q", f32, (dh,), dev), _p(g["dw_k"], "dw_k", f32, (dh,), dev),
            B, T, Hq, Hkv, dh, dh if rot is None else rot, base, eps, io,
            _p(workspace, "workspace", None, None, dev),
            workspace.numel() * workspace.element_size(), st), "rglru_qk_norm_rope_bwd")
    return g


def rglru_local_attn_fwd(q, k, v, *, window=0, sinks=0, scale=None, lens=None, out=None, lse=None,
                         want_lse=True, dev_status=None, stream=None):
    """Attention of q (B, T, Hq, dh) over k, v (B, S, Hkv, dh): causal, the last `window` keys
    (0: all) and the first `sinks` keys; query t stands at position t + S - T. `scale` is
    1 / sqrt(dh) by default. With `lens` (B, int32; S == T) row b has lens[b] tokens, and rows
    past them are left as they were in given outputs, zeros (and -inf in lse) in ones allocated
    here. Returns (out, lse), lse (B, Hq, T) or None when it is neither wanted nor given."""
    views, dev, dt, io, B, T, S, Hq, Hkv, dh = _sizes(q, k, v)
    with _on(dev, stream) as st:
        if out is None:
            make = torch.empty if lens is None else torch.zeros
            out = make((B, T, Hq, dh), device=q.device, dtype=dt)
        if lse is None and want_lse:
            lse = torch.empty((B, Hq, T), device=q.device, dtype=torch.float32)
            if lens is not None:
                lse.fill_(float("-inf"))
        _check(LIB.rglru_local_attn_fwd(
            *views, _p(lens, "lens", torch.int32, (B,), dev, True),
            _p(out, "out", dt, (B, T, Hq, dh), dev),
            _p(lse, "lse", torch.float32, (B, Hq, T), dev, True), B, T, S, Hq, Hkv, dh,
            window, sinks, dh ** -0.5 if scale is None else scale, io,
            _p(dev_status, "dev_status", torch.int32, None, dev, True), st),
            "rglru_local_attn_fwd")
    return out, lse


def rglru_local_attn_bwd(q, k, v, out, lse, dout, *, window=0, sinks=0, scale=None, lens=None,
                         workspace=None, grads=None, dev_status=None, stream=None):
    """Backward of rglru_local_attn_fwd from its inputs, its out and lse, and dout. Returns a
    dict with dq, dk, dv (dense, the I/O dtype). `grads` may hold preallocated outputs by name;
    with `lens`, rows past a sequence are left as they were there, zeros otherwise."""
    views, dev, dt, io, B, T, S, Hq, Hkv, dh = _sizes(q, k, v)
    g = dict(grads or {})
    with _on(dev, stream) as st:
        make = torch.empty if lens is None else torch.zeros
        for name, shape in (("dq", (B, T, Hq, dh)), ("dk", (B, S, Hkv, dh)),
                            ("dv", (B, S, Hkv, dh))):
            if g.get(name) is None:
                g[name] = make(shape, device=q.device, dtype=dt)
        need = LIB.rglru_local_attn_bwd_workspace_bytes(B, T, S, Hq, Hkv, dh, window, sinks, io)
        workspace = _workspace(workspace, need, q.device)
        _check(LIB.rglru_local_attn_bwd(
            *views, _p(out, "out", dt, (B, T, Hq, dh), dev),
            _p(lse, "lse", torch.float32, (B, Hq, T), dev),
            _p(dout, "dout", dt, (B, T, Hq, dh), dev),
            _p(lens, "lens", torch.int32, (B,), dev, True),
            _p(g["dq"], "dq", dt, (B, T, Hq, dh), dev), _p(g["dk"], "dk", dt, (B, S, Hkv, dh), dev),
            _p(g["dv"], "dv", dt, (B, S, Hkv, dh), dev), B, T, S, Hq, Hkv, dh, window, sinks,
            dh ** -0.5 if scale is None else scale, io, _p(workspace, "workspace", None, None, dev),
            workspace.numel() * workspace.element_size(),
            _p(dev_status, "dev_status", torch.int32, None, dev, True), st),
            "rglru_local_attn_bwd")
    return g


def rglru_paged_attn_decode(q, k_cache, v_cache, page_table, lens, *, window=0, sinks=0,
                            scale=None, out=None, workspace=None, dev_status=None, stream=None):
    """Attention of one new token of each sequence, q (B, Hq, dh), over its paged cache (pages,
    page_size, Hkv, dh): its last `window` keys (0: all) and its first `sinks`, of lens[b] keys
    (the new token's own among them; 0: the row of out is zeros). Returns out (B, Hq, dh)."""
    qp = _p(q, "q", None, None, None)
    if q.dim() != 3:
        raise ValueError("q must be (B, Hq, dh)")
    B, Hq, dh = q.shape
    dt, dev = q.dtype, q.get_device()
    io = _io_of(dt)
    _place(k_cache, "k_cache", dev)
    Hkv = k_cache.shape[2] if k_cache.dim() == 4 else 0
    kc, vc, table, pages, page_size, max_pages = _cache(k_cache, v_cache, page_table, dt, B, Hkv,
                                                        dh, dev)
    with _on(dev, stream) as st:
        if out is None:
            out = q.new_empty((B, Hq, dh))
        need = LIB.rglru_paged_attn_decode_workspace_bytes(B, Hq, Hkv, dh, page_size, max_pages,
                                                           window, sinks, io)
        workspace = _workspace(workspace, need, q.device)
        _check(LIB.rglru_paged_attn_decode(
            qp, kc, vc, table, _p(lens, "lens", torch.int32, (B,), dev),
            _p(out, "out", dt, (B, Hq, dh), dev), pages, page_size, max_pages, B, Hq, Hkv, dh,
            window, sinks, dh ** -0.5 if scale is None else scale, io,
            _p(workspace, "workspace", None, None, dev),
            workspace.numel() * workspace.element_size(),
            _p(dev_status, "dev_status", torch.int32, None, dev, True), st),
            "rglru_paged_attn_decode")
    return out
