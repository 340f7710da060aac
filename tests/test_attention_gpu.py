"""GPU parity of the local attention operators against the float64 oracle
(oracle/attention_oracle.py).

Bars, elementwise, from the arithmetic. u = 2^-24 and ub = 2^-8 are half a step of fp32 and of
bf16, relative to the value. A sum of n fp32 products is off by at most (n + 2) u times the sum
of their absolute values; 2 u is allowed a step where the tensor core's accumulation may cut
instead of round.
 - Scores: e_s = 2 u (dh + 4) scale max_ij sum_d |q k|. A weight is then off by a factor
   e^(+-2 e_s) (its own score and its row's sum), and exp and the sums of up to n keys add
   (n + 16) u: w = 2 e_s + (n + 16) 2 u, relative.
 - out: w sum_j p_j |v_j|, and for bf16 ub sum_j p_j |v_j| (the weights are rounded for the
   product) + ub |out| (the store).
 - lse: e_s + (n + 16) 2 u + 4 u |lse|.
 - gradients: the terms of each are weights or score gradients times inputs. A weight is off by
   w (and the stored lse's own 2 u |lse|), dout . v and delta by 2 u (dh + 4) of their absolute
   terms, which the oracle carries through (`through`); the sums of m terms add 2 u (m + 4) of
   the absolute terms (`size`); bf16 adds ub size (weights and score gradients are rounded for
   the product) + ub |gradient|.
 - norms and rotation: 32 u of |n_i| + |n_j| (16 roundings in the norm's sum, root and products,
   the angle's 2 u pi, sine and cosine, the turn), + ub |y| in bf16. Their backward: the same
   through r (|g w| + |xhat| mean |g w xhat|), g of both of a pair, twice; dw: (64 + rows) u of
   sum |g xhat|.
"""
import numpy as np
import pytest
import torch

import gated_linear_recurrence_rglru_b200 as rg
from oracle import attention_oracle as orc

pytestmark = pytest.mark.gpu

U, UB = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(gen, shape, io, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(DT[io])


def close(got, ref, tol, what):
    got = f64(got)
    assert got.shape == ref.shape, what
    with np.errstate(invalid="ignore"):
        bad = ~np.isnan(ref) & ~(np.abs(got - ref) <= tol) & ~((got == ref) & np.isinf(ref))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {i}: got {got[i]}, "
                             f"expected {ref[i]}, allowed {np.broadcast_to(tol, ref.shape)[i]}")


def layout(t, kind, dev):
    """The same (B, T, H, dh) values on the device, dense, as a slice of wider rows, or head-major."""
    B, T, H, dh = t.shape
    if kind == "dense":
        return t.to(dev)
    if kind == "heads":
        return t.transpose(1, 2).contiguous().to(dev).transpose(1, 2)
    wide = torch.full((B + 1, T, 2 * H + 1, dh), float("nan"), dtype=t.dtype, device=dev)
    v = wide[:B, :, H:2 * H]
    v.copy_(t.to(dev))
    return v


# ------------------------------------------------------------------- norms and rotation

QK_CASES = [  # io, B, T, Hq, Hkv, dh, rot, layout, far, weights
    ("bf16", 2, 5, 10, 1, 256, 128, "slice", 0, True), ("bf16", 1, 1, 4, 4, 64, 64, "dense", 0, True),
    ("f32", 3, 7, 4, 2, 64, 32, "heads", 1000, True), ("f32", 1, 33, 3, 1, 128, 128, "slice", 2 ** 31 - 40, False),
    ("bf16", 2, 3, 5, 5, 8, 0, "dense", 0, True), ("f32", 2, 9, 7, 2, 72, 48, "slice", -50, True),
    ("bf16", 1, 700, 16, 4, 128, 128, "slice", 500000, True), ("f32", 1, 2, 33, 1, 256, 256, "dense", 7, True),
    ("bf16", 4, 250, 2, 1, 40, 16, "heads", 3, True), ("f32", 2, 2, 2, 2, 16, 16, "dense", 0, False),
]


def qk_inputs(io, B, T, Hq, Hkv, dh, far, weights, seed):
    gen = torch.Generator().manual_seed(seed)
    q, k = randn(gen, (B, T, Hq, dh), io), randn(gen, (B, T, Hkv, dh), io)
    q[0, 0, 0] = 0                                # a row of zeros: eps alone under the root
    w = [(1 + randn(gen, (dh,), "f32", 0.3)).to(DT[io]) if weights else None for _ in range(2)]
    first = far + torch.arange(B)[:, None] * 3
    return gen, q, k, w, (first + torch.arange(T)).to(torch.int32)


@pytest.mark.parametrize("case", QK_CASES, ids=str)
def test_qk_norm_rope_fwd(cuda_device, case):
    io, B, T, Hq, Hkv, dh, rot, kind, far, weights = case
    _, q, k, w, pos = qk_inputs(io, B, T, Hq, Hkv, dh, far, weights, 1)
    wd = [x.to(cuda_device) if x is not None else None for x in w]
    got = rg.rglru_qk_norm_rope_fwd(layout(q, kind, cuda_device), layout(k, kind, cuda_device), *wd,
                                    pos.to(cuda_device), rot=rot)
    for x, wx, y, name in ((q, w[0], got[0], "q"), (k, w[1], got[1], "k")):
        check_norm(y, x, wx, pos, rot, io, name)


def check_norm(y, x, w, pos, rot, io, name):
    w = f64(w) if w is not None else None
    ref = orc.qk_norm_rope(f64(x), w, pos.numpy(), rot, 10000.0, 1e-6)
    n = np.abs(orc.qk_norm_rope(f64(x), w, pos.numpy() * 0, rot, 10000.0, 1e-6))
    other = np.concatenate([n[..., rot // 2:rot], n[..., :rot // 2], 0 * n[..., rot:]], -1)
    close(y, ref, 32 * U * (n + other) + (UB * np.abs(ref) if io == "bf16" else 0), name)


def test_qk_norm_rope_default_positions(cuda_device):
    _, q, k, w, _ = qk_inputs("bf16", 2, 19, 4, 1, 64, 0, True, 2)
    pos = torch.arange(19, dtype=torch.int32).repeat(2, 1).to(cuda_device)
    a = [x.to(cuda_device) for x in (q, k, *w)]
    for x, y in zip(rg.rglru_qk_norm_rope_fwd(*a), rg.rglru_qk_norm_rope_fwd(*a, pos, rot=64)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("case", QK_CASES, ids=str)
def test_qk_norm_rope_bwd(cuda_device, case):
    io, B, T, Hq, Hkv, dh, rot, kind, far, weights = case
    gen, q, k, w, pos = qk_inputs(io, B, T, Hq, Hkv, dh, far, weights, 3)
    q[0, 0, 0] = randn(gen, (dh,), io)            # (at zero the gradient is 1 / sqrt(eps): huge)
    dq, dk = randn(gen, q.shape, io), randn(gen, k.shape, io)
    wd = [x.to(cuda_device) if x is not None else None for x in w]
    args = (layout(q, kind, cuda_device), layout(k, kind, cuda_device), dq.to(cuda_device),
            dk.to(cuda_device), *wd, pos.to(cuda_device))
    got = rg.rglru_qk_norm_rope_bwd(*args, rot=rot)
    for x, dy, wx, n in ((q, dq, w[0], "q"), (k, dk, w[1], "k")):
        x, dy, wx = f64(x), f64(dy), f64(wx) if wx is not None else None
        dx, dw = orc.qk_norm_rope_bwd(x, wx, dy, pos.numpy(), rot, 10000.0, 1e-6)
        g = np.abs(dy)
        g = g + np.concatenate([g[..., rot // 2:rot], g[..., :rot // 2], 0 * g[..., rot:]], -1)
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-6)
        xh, gw = np.abs(x * r), g * np.abs(1 if wx is None else wx)
        close(got["d" + n], dx, 64 * U * r * (gw + xh * np.mean(gw * xh, -1, keepdims=True))
              + (UB * np.abs(dx) if io == "bf16" else 0), "d" + n)
        rows = x.shape[0] * x.shape[1] * x.shape[2]
        close(got["dw_" + n], dw, (64 + rows) * U * (g * xh).sum((0, 1, 2)), "dw_" + n)
    again = rg.rglru_qk_norm_rope_bwd(*args, rot=rot)
    assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("io,B,T,Hq,Hkv,dh,page", [
    ("bf16", 3, 1, 10, 1, 256, 16), ("f32", 2, 7, 4, 2, 64, 5), ("bf16", 4, 3, 2, 2, 40, 1)])
def test_qk_norm_rope_append(cuda_device, io, B, T, Hq, Hkv, dh, page):
    gen, q, k, w, _ = qk_inputs(io, B, T, Hq, Hkv, dh, 0, True, 4)
    v = randn(gen, k.shape, io)
    most = 40 // page + 1
    table = torch.randperm(B * most + 3, generator=gen)[:B * most].view(B, most).to(torch.int32)
    pos = (torch.arange(B)[:, None] * 11 + torch.arange(T)).to(torch.int32)
    pos[B - 1, T - 1] = -1                          # padding
    bad = (0, 0)                                    # a page out of range: reported, not written
    table[bad[0], int(pos[bad]) // page] = B * most + 3
    kc, vc = randn(gen, (B * most + 3, page, Hkv, dh), io), randn(gen, (B * most + 3, page, Hkv, dh), io)
    d = [x.to(cuda_device) for x in (kc, vc, table, pos, *w)]
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    got = rg.rglru_qk_norm_rope_append(
        *[layout(x, "slice", cuda_device) for x in (q, k, v)], *d, rot=dh // 16 * 16,
        dev_status=status)
    rot = dh // 16 * 16
    on = pos >= 0
    check_norm(got[on.to(cuda_device)][None], q[on][None], w[0], pos[on][None], rot, io, "q")
    assert torch.all(got[~on.to(cuda_device)] == 0)
    assert int(status) == 1
    kept = [(b, t) for b in range(B) for t in range(T)
            if on[b, t] and not (b == 0 and int(pos[b, t]) // page == int(pos[bad]) // page)]
    slots = [(int(table[b, int(pos[b, t]) // page]), int(pos[b, t]) % page) for b, t in kept]
    if kept:
        pick = tuple(torch.tensor(x) for x in zip(*slots))
        rows = tuple(torch.tensor(x) for x in zip(*kept))
        check_norm(d[0].cpu()[pick][None], k[rows][None], w[1], pos[rows][None], rot, io, "k_cache")
        assert torch.equal(d[1].cpu()[pick], v[rows])
        kc[pick], vc[pick] = d[0].cpu()[pick], d[1].cpu()[pick]
    assert torch.equal(d[0].cpu(), kc) and torch.equal(d[1].cpu(), vc)    # nothing else changed


# ------------------------------------------------------------------- windowed attention

ATTN_CASES = [  # io, B, T, S, Hq, Hkv, dh, window, sinks, lens, layout
    ("bf16", 1, 1, 1, 1, 1, 64, 0, 0, None, "dense"),
    ("bf16", 2, 300, 300, 4, 2, 64, 0, 0, None, "slice"),
    ("bf16", 1, 513, 513, 2, 1, 128, 100, 0, None, "slice"),
    ("bf16", 1, 400, 400, 3, 1, 256, 129, 5, None, "slice"),
    ("bf16", 1, 130, 700, 2, 2, 128, 200, 3, None, "heads"),
    ("bf16", 2, 70, 33, 2, 1, 64, 0, 0, None, "dense"),          # queries that see no key
    ("bf16", 3, 260, 260, 4, 4, 64, 64, 1, [260, 0, 131], "slice"),
    ("bf16", 3, 200, 200, 2, 1, 256, 0, 0, [1, 129, 200], "slice"),
    ("bf16", 2, 384, 384, 5, 1, 128, 130, 200, [384, 255], "heads"),  # sinks over several tiles
    ("bf16", 1, 20, 1000, 4, 1, 256, 37, 0, None, "dense"),      # keys that no query sees
    ("bf16", 1, 257, 257, 1, 1, 64, 1, 0, None, "dense"),        # every query sees itself alone
    ("f32", 2, 100, 100, 4, 2, 64, 0, 0, None, "slice"),
    ("f32", 3, 1, 1, 4, 2, 128, 0, 0, None, "dense"), ("f32", 1, 40, 40, 1, 1, 64, 1, 0, None, "dense"),
    ("bf16", 2, 1, 1, 4, 1, 256, 1024, 4, None, "dense"), ("bf16", 1, 3, 3, 2, 1, 128, 2, 0, None, "dense"),
    ("f32", 1, 70, 200, 2, 1, 128, 60, 3, None, "heads"),
    ("f32", 2, 90, 90, 3, 1, 256, 33, 2, [90, 17], "slice"),
    ("f32", 1, 50, 20, 2, 2, 192, 5, 1, None, "dense"),
    ("bf16", 2, 77, 77, 2, 1, 72, 20, 1, None, "slice"),
    ("f32", 1, 65, 65, 1, 1, 8, 0, 0, None, "dense"),
    # few rows, many keys: a cluster of blocks takes a query tile's keys
    ("bf16", 1, 128, 4096, 4, 2, 128, 0, 0, None, "dense"),
    ("bf16", 1, 3, 2500, 3, 3, 64, 0, 0, None, "slice"),
    ("bf16", 2, 200, 1500, 3, 1, 64, 700, 130, None, "slice"),
    ("bf16", 1, 16, 1030, 4, 1, 256, 0, 0, None, "heads"),
    ("bf16", 1, 1, 3000, 5, 1, 256, 2000, 0, None, "dense"),
    ("bf16", 3, 1000, 1000, 1, 1, 64, 0, 0, [1000, 0, 300], "slice"),
    ("bf16", 2, 640, 640, 2, 2, 128, 400, 3, [640, 129], "heads"),
    ("bf16", 1, 600, 500, 2, 1, 128, 0, 0, None, "dense"),
]


def attn_inputs(case, seed, dev):
    io, B, T, S, Hq, Hkv, dh, window, sinks, lens, kind = case
    gen = torch.Generator().manual_seed(seed)
    q, k, v = (randn(gen, s, io) for s in ((B, T, Hq, dh), (B, S, Hkv, dh), (B, S, Hkv, dh)))
    hidden = torch.zeros(B, S, dtype=torch.bool)
    if lens is None:
        hidden[:] = torch.tensor(~orc.visible(T, S, window, sinks).any(0))
    else:
        hidden[:] = torch.arange(S) >= torch.tensor(lens)[:, None]
    k[hidden], v[hidden] = float("nan"), float("inf")     # what no query sees may hold anything
    if lens is not None:
        q[hidden] = float("nan")
    dl = torch.tensor(lens, dtype=torch.int32, device=dev) if lens is not None else None
    return gen, (q, k, v), [layout(x, kind, dev) for x in (q, k, v)], dl


def score_error(q, k, dh, scale):
    a, b = np.abs(np.nan_to_num(f64(q))), np.abs(np.nan_to_num(f64(k)))
    return 2 * U * (dh + 4) * scale * np.sqrt((a * a).sum(-1).max() * (b * b).sum(-1).max())


@pytest.mark.parametrize("case", ATTN_CASES, ids=str)
def test_local_attn_fwd(cuda_device, case):
    io, B, T, S, Hq, Hkv, dh, window, sinks, lens, _ = case
    _, (q, k, v), d, dl = attn_inputs(case, 11, cuda_device)
    scale = dh ** -0.5
    out = torch.full((B, T, Hq, dh), 7.0, dtype=DT[io], device=cuda_device)
    lse = torch.full((B, Hq, T), 7.0, device=cuda_device)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    rg.rglru_local_attn_fwd(*d, window=window, sinks=sinks, lens=dl, out=out, lse=lse, dev_status=status)
    assert int(status) == 0
    ref, lref, size = orc.local_attn(f64(q), f64(k), f64(v), window, sinks, scale, lens)
    es = score_error(q, k, dh, scale)
    w = 2 * es + (S + 16) * 2 * U
    close(out, ref, w * size + (UB * (size + np.abs(ref)) if io == "bf16" else 0), "out")
    close(lse, lref, es + (S + 16) * 2 * U + 4 * U * np.abs(np.nan_to_num(lref, neginf=0)), "lse")
    if lens is not None:
        for b, n in enumerate(lens):                # rows past a sequence: left as they were
            assert torch.all(out[b, n:] == 7) and torch.all(lse[b, :, n:] == 7)
    out2, none = rg.rglru_local_attn_fwd(*d, window=window, sinks=sinks, lens=dl, want_lse=False)
    assert none is None
    keep = ~torch.isnan(torch.tensor(ref)).to(cuda_device)
    assert torch.equal(out2[keep], out[keep])


@pytest.mark.parametrize("case", ATTN_CASES, ids=str)
def test_local_attn_bwd(cuda_device, case):
    io, B, T, S, Hq, Hkv, dh, window, sinks, lens, _ = case
    gen, (q, k, v), d, dl = attn_inputs(case, 12, cuda_device)
    scale = dh ** -0.5
    ref, lref, _ = orc.local_attn(f64(q), f64(k), f64(v), window, sinks, scale, lens)
    out, lse = torch.tensor(ref).to(DT[io]), torch.tensor(lref).float()
    dout = randn(gen, q.shape, io)
    if lens is not None:
        dout[torch.arange(T) >= torch.tensor(lens)[:, None]] = float("nan")
    grads = {n: torch.full((B, s, h, dh), 7.0, dtype=DT[io], device=cuda_device)
             for n, s, h in (("dq", T, Hq), ("dk", S, Hkv), ("dv", S, Hkv))}
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    args = (*d, out.to(cuda_device), lse.to(cuda_device), dout.to(cuda_device))
    got = rg.rglru_local_attn_bwd(*args, window=window, sinks=sinks, lens=dl, grads=grads, dev_status=status)
    assert int(status) == 0 and all(got[n] is grads[n] for n in grads)
    # queries that see few keys do not take the row sums of dout and out from the stored out
    pos = np.arange(T) + S - T
    few = (pos < 16) | (0 < window <= 16 - sinks)
    given = np.where(few[None, :, None, None], ref, f64(out))
    g, size, through = orc.local_attn_bwd(f64(q), f64(k), f64(v), given, f64(dout), window, sinks,
                                          scale, lens)
    w = 2 * score_error(q, k, dh, scale) + 32 * U + 2 * U * np.abs(np.nan_to_num(lref, neginf=0)).max()
    for n in grads:
        terms = (S if n == "dq" else T * Hq // Hkv) + 4
        tol = w * (size[n] + through[n]) + 2 * U * (dh + 4) * through[n] + 2 * U * terms * size[n]
        close(got[n], g[n], tol + (UB * (size[n] + np.abs(g[n])) if io == "bf16" else 0), n)
    if lens is not None:
        for b, m in enumerate(lens):
            assert all(torch.all(got[n][b, m:] == 7) for n in grads)
    # a query that sees one key has a constant softmax: exactly no gradient of its scores
    if lens is None and np.any(pos == 0):
        assert torch.all(got["dq"][:, int(np.argmax(pos == 0))] == 0)
    if (window == 1 and sinks == 0) or S == T == 1:
        assert torch.all(got["dq"] == 0) and torch.all(got["dk"] == 0)
    again = rg.rglru_local_attn_bwd(*args, window=window, sinks=sinks, lens=dl)
    if lens is None:
        assert all(torch.equal(got[n], again[n]) for n in grads)
    else:
        assert all(torch.equal(got[n][b, :m], again[n][b, :m]) for n in grads for b, m in enumerate(lens))


@pytest.mark.parametrize("io,dh,T,G", [("bf16", 64, 300, 2), ("bf16", 64, 700, 2), ("bf16", 128, 40, 1),
                                       ("bf16", 128, 1100, 1), ("bf16", 256, 200, 2),
                                       ("f32", 64, 90, 2), ("f32", 256, 40, 1)])
def test_nan_reaches_who_sees_it_alone(cuda_device, io, dh, T, G):
    """A NaN in a query is that query's output; a NaN in a key that of the queries that see it."""
    gen = torch.Generator().manual_seed(61)
    q, k, v = (randn(gen, (1, T, h, dh), io).to(cuda_device) for h in (2, 2 // G, 2 // G))
    out, lse = rg.rglru_local_attn_fwd(q, k, v)
    q2, k2 = q.clone(), k.clone()
    q2[0, 5, 1, 3] = float("nan")
    got, glse = rg.rglru_local_attn_fwd(q2, k, v)
    assert torch.isnan(got[0, 5, 1]).all() and torch.isnan(glse[0, 1, 5])
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[0, 5, 1] = False
    assert torch.equal(got[keep], out[keep]) and int(torch.isnan(glse).sum()) == 1
    k2[0, 20, 0, 0] = float("nan")
    got, glse = rg.rglru_local_attn_fwd(q, k2, v)
    assert torch.equal(got[:, :20], out[:, :20]) and torch.equal(glse[..., :20], lse[..., :20])
    assert torch.isnan(got[:, 20:, 0]).all() and torch.isnan(glse[:, 0, 20:]).all()


@pytest.mark.parametrize("io,dh,T,S,window,sinks", [("bf16", 64, 16, 16, 0, 0), ("bf16", 256, 4, 7, 0, 0),
                                                    ("bf16", 128, 40, 40, 9, 7), ("bf16", 72, 30, 30, 16, 0),
                                                    ("f32", 64, 10, 5, 0, 0)])
def test_rounding_of_out_stays_out_of_rows_with_few_keys(cuda_device, io, dh, T, S, window, sinks):
    """Queries that see up to 16 keys get their gradients from the keys: another rounding of out
    changes no bit."""
    gen = torch.Generator().manual_seed(71)
    q, k, v, dout = (randn(gen, (2, n, h, dh), io).to(cuda_device) for n, h in ((T, 4), (S, 2), (S, 2), (T, 4)))
    out, lse = rg.rglru_local_attn_fwd(q, k, v, window=window, sinks=sinks)
    g = rg.rglru_local_attn_bwd(q, k, v, out, lse, dout, window=window, sinks=sinks)
    other = out * (1 + 2 * torch.finfo(out.dtype).eps)
    assert not torch.equal(out, other)
    again = rg.rglru_local_attn_bwd(q, k, v, other, lse, dout, window=window, sinks=sinks)
    assert all(torch.equal(g[n], again[n]) for n in g)


# ---------------------------------------------------------------- one token over a cache

DECODE_CASES = [  # io, Hq, Hkv, dh, page, lens, window, sinks, max_pages
    ("bf16", 10, 1, 256, 16, [1, 700, 0, 33], 0, 0, 50), ("bf16", 4, 4, 64, 64, [257], 0, 0, 8),
    ("bf16", 16, 4, 128, 16, [1000, 999], 100, 3, 64), ("bf16", 40, 2, 64, 3, [50, 64], 0, 0, 22),
    ("bf16", 8, 1, 128, 32, [5000], 0, 0, 160), ("bf16", 2, 1, 256, 16, [2049, 4], 1024, 4, 400),
    ("f32", 4, 4, 64, 16, [1, 0, 300], 0, 0, 32), ("f32", 10, 1, 256, 5, [333, 40], 64, 2, 70),
    ("f32", 3, 1, 128, 16, [3000], 0, 0, 200), ("bf16", 6, 2, 72, 7, [100, 29], 0, 0, 16),
    ("f32", 2, 2, 8, 1, [40, 1], 7, 50, 40),
]


def decode_inputs(case, seed):
    io, Hq, Hkv, dh, page, lens, window, sinks, most = case
    gen = torch.Generator().manual_seed(seed)
    B, pages = len(lens), len(lens) * most + 2
    table = torch.randperm(pages, generator=gen)[:B * most].view(B, most).to(torch.int32)
    kc, vc = (torch.full((pages, page, Hkv, dh), float("nan"), dtype=DT[io]) for _ in range(2))
    for b, n in enumerate(lens):                    # only what is visible holds numbers
        used = set()
        for j in range(n):
            if window == 0 or j > n - 1 - window or j < sinks:
                p = int(table[b, j // page])
                used.add(j // page)
                kc[p, j % page], vc[p, j % page] = randn(gen, (Hkv, dh), io), randn(gen, (Hkv, dh), io)
        for x in set(range(most)) - used:           # a page without visible keys may be absent
            table[b, x] = -1
    return randn(gen, (B, Hq, dh), io), kc, vc, table, torch.tensor(lens, dtype=torch.int32)


@pytest.mark.parametrize("case", DECODE_CASES, ids=str)
def test_paged_attn_decode(cuda_device, case):
    io, Hq, Hkv, dh, page, lens, window, sinks, most = case
    host = decode_inputs(case, 21)
    d = [x.to(cuda_device) for x in host]
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    out = torch.full((len(lens), Hq, dh), 7.0, dtype=DT[io], device=cuda_device)
    got = rg.rglru_paged_attn_decode(*d, window=window, sinks=sinks, out=out, dev_status=status)
    assert int(status) == 0 and got is out
    scale = dh ** -0.5
    ref, size = orc.paged_decode(*[f64(x) for x in host[:3]], host[3].numpy(), lens, window, sinks, scale)
    w = 2 * score_error(host[0], host[1], dh, scale) + (max(lens) + 16) * 2 * U
    close(got, ref, w * size + (UB * (size + np.abs(ref)) if io == "bf16" else 0), "out")
    assert torch.equal(rg.rglru_paged_attn_decode(*d, window=window, sinks=sinks), got)


@pytest.mark.parametrize("io,dh,lens", [("bf16", 128, [60, 3000]), ("bf16", 256, [60, 50]), ("f32", 64, [60, 9000])])
def test_paged_attn_decode_nan(cuda_device, io, dh, lens):
    case = (io, 4, 2, dh, 16, lens, 0, 0, max(lens) // 16 + 1)
    d = [x.to(cuda_device) for x in decode_inputs(case, 23)]
    out = rg.rglru_paged_attn_decode(*d)
    q = d[0].clone()
    q[1, 2, 0] = float("nan")
    got = rg.rglru_paged_attn_decode(q, *d[1:])
    assert torch.isnan(got[1, 2]).all()
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1, 2] = False
    assert torch.equal(got[keep], out[keep])


@pytest.mark.parametrize("io,dh", [("bf16", 128), ("f32", 64)])
def test_paged_attn_decode_bad_pages_are_hidden(cuda_device, io, dh):
    case = (io, 4, 2, dh, 8, [30, 45], 0, 0, 4)
    q, kc, vc, table, lens = decode_inputs((io, 4, 2, dh, 8, [30, 32], 0, 0, 4), 22)
    table[0, 1], table[1, 3] = kc.shape[0], -5
    lens[1] = case[5][1]                            # past what its table can name: cut to 32
    d = [x.to(cuda_device) for x in (q, kc, vc, table, lens)]
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    got = rg.rglru_paged_attn_decode(*d, dev_status=status)
    assert int(status) == 1
    keep = [[j for j in range(30) if j // 8 != 1], list(range(24))]
    for b, keys in enumerate(keep):
        at = [(int(table[b, j // 8]), j % 8) for j in keys]
        k, v = (np.stack([f64(c[p, s]) for p, s in at])[None] for c in (kc, vc))
        ref, size = orc.paged_decode(f64(q[b:b + 1]), k, v, np.zeros((1, 1), int), [len(keys)], 0, 0, dh ** -0.5)
        w = 2 * score_error(q, torch.tensor(k), dh, dh ** -0.5) + 64 * 2 * U
        close(got[b:b + 1], ref, w * size + (UB * (size + np.abs(ref)) if io == "bf16" else 0), b)


# ------------------------------------------------------------------------- used together

@pytest.mark.parametrize("io,Hq,Hkv,dh,window,sinks", [
    ("bf16", 10, 1, 256, 16, 2), ("bf16", 4, 2, 64, 0, 0), ("f32", 4, 4, 64, 12, 0)])
def test_prompt_then_steps(cuda_device, io, Hq, Hkv, dh, window, sinks):
    """A prompt through the norm, the rotation and the windowed attention while its keys fill a
    paged cache, then single tokens through the cache: the same as one pass over all tokens."""
    B, T, P, page = 2, 45, 37, 8
    gen, q, k, w, pos = qk_inputs(io, B, T, Hq, Hkv, dh, 0, True, 31)
    v = randn(gen, k.shape, io)
    pos = torch.arange(T, dtype=torch.int32).repeat(B, 1)
    q, k, v, pos, wq, wk = (x.to(cuda_device) for x in (q, k, v, pos, *w))
    most = T // page + 1
    table = torch.randperm(B * most, generator=gen).view(B, most).to(torch.int32).to(cuda_device)
    cache = [torch.full((B * most, page, Hkv, dh), float("nan"), dtype=DT[io], device=cuda_device)
             for _ in range(2)]
    qn, kn = rg.rglru_qk_norm_rope_fwd(q, k, wq, wk, pos)
    whole, _ = rg.rglru_local_attn_fwd(qn, kn, v, window=window, sinks=sinks)
    qp = rg.rglru_qk_norm_rope_append(q[:, :P], k[:, :P], v[:, :P], *cache, table,
                                      pos[:, :P].contiguous(), wq, wk)
    assert torch.equal(qp, qn[:, :P])
    first, _ = rg.rglru_local_attn_fwd(qp, kn[:, :P], v[:, :P], window=window, sinks=sinks)
    got = [first]
    for t in range(P, T):
        qt = rg.rglru_qk_norm_rope_append(q[:, t:t + 1], k[:, t:t + 1], v[:, t:t + 1], *cache, table,
                                          pos[:, t:t + 1].contiguous(), wq, wk)
        lens = torch.full((B,), t + 1, dtype=torch.int32, device=cuda_device)
        got.append(rg.rglru_paged_attn_decode(qt[:, 0], *cache, table, lens, window=window,
                                              sinks=sinks)[:, None])
    got = torch.cat(got, 1)
    # both sides hold the bars of the header against the exact values
    ref, _, size = orc.local_attn(f64(qn), f64(kn), f64(v), window, sinks, dh ** -0.5)
    w = 2 * score_error(qn, kn, dh, dh ** -0.5) + (T + 16) * 2 * U
    tol = w * size + (UB * (size + np.abs(ref)) if io == "bf16" else 0)
    close(got, ref, tol, "steps")
    close(whole, ref, tol, "whole")


def test_training_step_by_differences(cuda_device):
    """Norm, rotation and attention together in fp32: the chained gradients against central
    differences of the float64 oracle in random directions. The gradients' own errors are of the
    order 1e-5 of their size (the bars above), the differences' 1e-6; 1e-3 is asked."""
    B, T, Hq, Hkv, dh, window, sinks = 2, 21, 4, 2, 64, 9, 1
    gen, q, k, w, pos = qk_inputs("f32", B, T, Hq, Hkv, dh, 5, True, 41)
    q[0, 0, 0] = randn(gen, (dh,), "f32")
    v, dout = randn(gen, k.shape, "f32"), randn(gen, q.shape, "f32")
    d = [x.to(cuda_device) for x in (q, k, v, *w, pos, dout)]
    qn, kn = rg.rglru_qk_norm_rope_fwd(d[0], d[1], d[3], d[4], d[5])
    out, lse = rg.rglru_local_attn_fwd(qn, kn, d[2], window=window, sinks=sinks)
    g = rg.rglru_local_attn_bwd(qn, kn, d[2], out, lse, d[6], window=window, sinks=sinks)
    gn = rg.rglru_qk_norm_rope_bwd(d[0], d[1], g["dq"], g["dk"], d[3], d[4], d[5])
    x = dict(dq=f64(q), dk=f64(k), dv=f64(v), dw_q=f64(w[0]), dw_k=f64(w[1]))
    grads = dict(dq=gn["dq"], dk=gn["dk"], dv=g["dv"], dw_q=gn["dw_q"], dw_k=gn["dw_k"])

    def loss(x):
        a = orc.qk_norm_rope(x["dq"], x["dw_q"], pos.numpy(), dh, 10000.0, 1e-6)
        b = orc.qk_norm_rope(x["dk"], x["dw_k"], pos.numpy(), dh, 10000.0, 1e-6)
        return (orc.local_attn(a, b, x["dv"], window, sinks, dh ** -0.5)[0] * f64(dout)).sum()

    rng = np.random.default_rng(5)
    for n in x:
        for _ in range(3):
            step = rng.standard_normal(x[n].shape)
            e = 1e-5
            diff = (loss({**x, n: x[n] + e * step}) - loss({**x, n: x[n] - e * step})) / (2 * e)
            got = (f64(grads[n]) * step).sum()
            size = np.sqrt((f64(grads[n]) ** 2).sum())
            assert abs(got - diff) <= 1e-3 * size, (n, got, diff, size)


def test_other_streams_and_graphs(cuda_device):
    """Each operator on a stream of the caller's, two at once, and captured and replayed on new
    inputs: the same bits as a plain call."""
    case = ("bf16", 2, 200, 200, 4, 2, 64, 50, 1, None, "dense")
    _, _, (q, k, v), _ = attn_inputs(case, 51, cuda_device)
    dout = torch.randn_like(q)
    dec = [x.to(cuda_device) for x in decode_inputs(("bf16", 4, 2, 64, 16, [3000, 77], 0, 0, 200), 52)]

    def calls(q, k, v, stream=None):
        qn, kn = rg.rglru_qk_norm_rope_fwd(q, k, stream=stream)
        out, lse = rg.rglru_local_attn_fwd(qn, kn, v, window=50, sinks=1, stream=stream)
        g = rg.rglru_local_attn_bwd(qn, kn, v, out, lse, dout, window=50, sinks=1, stream=stream)
        h = rg.rglru_qk_norm_rope_bwd(q, k, g["dq"], g["dk"], stream=stream)
        return [qn, kn, out, lse, *g.values(), *h.values(),
                rg.rglru_paged_attn_decode(*dec, stream=stream)]

    ref = [x.clone() for x in calls(q, k, v)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    both = [calls(q, k, v, s) for s in streams]
    torch.cuda.synchronize()
    for got in both:
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    held = [torch.randn_like(x) for x in (q, k, v)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(*held)
    for x, y in zip(held, (q, k, v)):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_refusals_of_the_binding(cuda_device):
    q = torch.zeros(2, 4, 4, 64, device=cuda_device)
    k = torch.zeros(2, 4, 2, 64, device=cuda_device)
    with pytest.raises(ValueError):                          # a broadcast head dimension is refused
        try:
            rg.rglru_local_attn_fwd(q, k[:, :, :1].expand(2, 4, 2, 64), k)
        except rg.RGLRUError as e:
            raise ValueError(str(e))
    with pytest.raises(TypeError):
        rg.rglru_local_attn_fwd(q, k.bfloat16(), k)
    with pytest.raises(TypeError):
        rg.rglru_local_attn_fwd(q.half(), k.half(), k.half())
    with pytest.raises(ValueError):
        rg.rglru_local_attn_fwd(q, k, k[:, :3])
    with pytest.raises(ValueError):
        rg.rglru_local_attn_fwd(q.transpose(2, 3), k, k)
    with pytest.raises(ValueError):
        rg.rglru_qk_norm_rope_fwd(q, k[:1])
    with pytest.raises(rg.RGLRUError):
        rg.rglru_qk_norm_rope_fwd(q, k, rot=72)
    with pytest.raises(rg.RGLRUError):
        rg.rglru_local_attn_fwd(q, k, k, window=-1)
    with pytest.raises(TypeError):
        rg.rglru_paged_attn_decode(q[:, 0].contiguous(), k, k, torch.zeros(2, 4, device=cuda_device),
                                   torch.zeros(2, dtype=torch.int32, device=cuda_device))
