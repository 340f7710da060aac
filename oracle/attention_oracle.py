"""Float64 definition of the local attention operators (include/rglru_attn.h), plain and
slow, one loop a batch row and head. It shares no code with the CUDA side.

Beside each result it can give an error scale: the sum of the absolute values of the terms
that the result adds up, which is what a rounding of the terms is relative to.
"""
from __future__ import annotations

import numpy as np


def rotation(x, positions, rot, base, back=False):
    """Turns the pairs (x[..., i], x[..., i + rot/2]) of (B, T, H, dh) by positions * base^(-2i/rot)."""
    y = np.array(x, dtype=np.float64)
    half = rot // 2
    for i in range(half):
        a = np.asarray(positions, dtype=np.float64) * base ** (-2.0 * i / rot)
        c, s = np.cos(a)[:, :, None], np.sin(a)[:, :, None]
        if back:
            s = -s
        y[..., i] = x[..., i] * c - x[..., i + half] * s
        y[..., i + half] = x[..., i + half] * c + x[..., i] * s
    return y


def qk_norm_rope(x, w, positions, rot, base, eps):
    x = np.asarray(x, dtype=np.float64)
    n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    if w is not None:
        n = n * np.asarray(w, dtype=np.float64)
    return rotation(n, positions, rot, base)


def qk_norm_rope_bwd(x, w, dy, positions, rot, base, eps):
    """(dx, dw) by the chain rule."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, dtype=np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    g = rotation(dy, positions, rot, base, back=True)
    dw = np.sum(g * x * r, axis=(0, 1, 2))
    gw = g * w
    return r * (gw - x * r * r * np.mean(gw * x, -1, keepdims=True)), dw


def visible(T, S, window, sinks):
    """(T, S): whether query t, at position t + S - T, sees key j."""
    pos = np.arange(T)[:, None] + (S - T)
    j = np.arange(S)[None, :]
    ok = j <= pos
    if window > 0:
        ok &= (j > pos - window) | (j < sinks)
    return ok


def _softmax(s, ok):
    s = np.where(ok, s, -np.inf)
    m = np.max(s, -1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    e = np.where(ok, np.exp(s - m), 0.0)
    l = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (np.log(l) + m)[..., 0]
    return e / np.where(l > 0, l, 1.0), lse


def local_attn(q, k, v, window, sinks, scale, lens=None):
    """out (B, T, Hq, dh), lse (B, Hq, T), and sum_j p_j |v_j|. Rows past lens are NaN."""
    B, T, Hq, dh = q.shape
    S, Hkv = k.shape[1], k.shape[2]
    out = np.full((B, T, Hq, dh), np.nan)
    size = np.full((B, T, Hq, dh), np.nan)
    lse = np.full((B, Hq, T), np.nan)
    for b in range(B):
        t, s = (T, S) if lens is None else (lens[b], lens[b])
        if t == 0:
            continue
        ok = visible(t, s, window, sinks)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            z = np.where(ok, scale * (q[b, :t, h] @ np.where(ok.any(0)[:, None], k[b, :s, g], 0).T), 0)
            p, lse[b, h, :t] = _softmax(z, ok)
            vv = np.where(ok.any(0)[:, None], v[b, :s, g], 0)
            out[b, :t, h] = p @ vv
            size[b, :t, h] = p @ np.abs(vv)
    return out, lse, size


def local_attn_bwd(q, k, v, out, dout, window, sinks, scale, lens=None):
    """Gradients with delta = rowsum(dout * out) from the given out, and for each the sum of the
    absolute terms, and the absolute terms that an error of the scores and of dout . v reaches
    through: dicts dq, dk, dv / sizes / through."""
    B, T, Hq, dh = q.shape
    S, Hkv = k.shape[1], k.shape[2]
    shapes = dict(dq=(B, T, Hq, dh), dk=(B, S, Hkv, dh), dv=(B, S, Hkv, dh))
    g = {n: np.full(s, np.nan) for n, s in shapes.items()}
    size = {n: np.zeros(s) for n, s in shapes.items()}
    through = {n: np.zeros(s) for n, s in shapes.items()}
    for b in range(B):
        t, s = (T, S) if lens is None else (lens[b], lens[b])
        g["dk"][b, :s] = g["dv"][b, :s] = 0.0
        if t == 0:
            continue
        ok = visible(t, s, window, sinks)
        seen = ok.any(0)[:, None]
        for h in range(Hq):
            c = h // (Hq // Hkv)
            qq, do = q[b, :t, h], dout[b, :t, h]
            kk, vv = np.where(seen, k[b, :s, c], 0), np.where(seen, v[b, :s, c], 0)
            p, _ = _softmax(np.where(ok, scale * (qq @ kk.T), 0), ok)
            ds = p * (do @ vv.T - (do * out[b, :t, h]).sum(-1, keepdims=True)) * scale
            # what an error of 1 in |dout| . |v| (and in delta) comes to
            ab = p * (np.abs(do) @ np.abs(vv).T + (np.abs(do) * np.abs(out[b, :t, h])).sum(-1, keepdims=True)) * scale
            g["dq"][b, :t, h] = ds @ kk
            g["dk"][b, :s, c] += ds.T @ qq
            g["dv"][b, :s, c] += p.T @ do
            size["dq"][b, :t, h] = np.abs(ds) @ np.abs(kk)
            size["dk"][b, :s, c] += np.abs(ds).T @ np.abs(qq)
            size["dv"][b, :s, c] += p.T @ np.abs(do)
            through["dq"][b, :t, h] = ab @ np.abs(kk)
            through["dk"][b, :s, c] += ab.T @ np.abs(qq)
            through["dv"][b, :s, c] += p.T @ np.abs(do)
    return g, size, through


def paged_decode(q, k_cache, v_cache, table, lens, window, sinks, scale):
    """out (B, Hq, dh) and sum_j p_j |v_j|."""
    B, Hq, dh = q.shape
    page, Hkv = k_cache.shape[1], k_cache.shape[2]
    out, size = np.zeros((B, Hq, dh)), np.zeros((B, Hq, dh))
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        keys = [j for j in range(n) if window == 0 or j > n - 1 - window or j < sinks]
        at = [(int(table[b, j // page]), j % page) for j in keys]
        k = np.stack([k_cache[p, s] for p, s in at])
        v = np.stack([v_cache[p, s] for p, s in at])
        for h in range(Hq):
            c = h // (Hq // Hkv)
            z = scale * (k[:, c] @ q[b, h])
            p = np.exp(z - z.max())
            p /= p.sum()
            out[b, h], size[b, h] = p @ v[:, c], p @ np.abs(v[:, c])
    return out, size
