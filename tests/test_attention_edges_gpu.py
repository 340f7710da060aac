"""GPU tests of the local attention operators where they are easily wrong: numbers that are not
finite, rows that see nothing, sizes at the ends of what is accepted, and calls large enough for
every block to take several units of work. The bars are those of test_attention_gpu.py.
"""
import numpy as np
import pytest
import torch

import gated_linear_recurrence_rglru_b200 as rg
import test_attention_gpu as base
from oracle import attention_oracle as orc
from test_attention_gpu import DT, U, UB, close, f64, randn

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- norms and rotation

def check_norm_grads(got, x, dy, w, pos, rot, io, eps, n):
    """dx and dw of one of q and k, within the bars of test_qk_norm_rope_bwd."""
    x, dy, w = f64(x), f64(dy), f64(w) if w is not None else None
    dx, dw = orc.qk_norm_rope_bwd(x, w, dy, pos.numpy(), rot, 10000.0, eps)
    g = np.abs(dy)
    g = g + np.concatenate([g[..., rot // 2:rot], g[..., :rot // 2], 0 * g[..., rot:]], -1)
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    xh, gw = np.abs(x * r), g * np.abs(1 if w is None else w)
    close(got["d" + n], dx, 64 * U * r * (gw + xh * np.mean(gw * xh, -1, keepdims=True))
          + (UB * np.abs(dx) if io == "bf16" else 0), "d" + n)
    rows = x.shape[0] * x.shape[1] * x.shape[2]
    close(got["dw_" + n], dw, (64 + rows) * U * (g * xh).sum((0, 1, 2)), "dw_" + n)


@pytest.mark.parametrize("io,B,T,Hq,Hkv,dh", [("bf16", 2, 9, 10, 1, 64), ("f32", 2, 9, 3, 1, 128),
                                              ("f32", 1, 5, 1, 1, 8), ("bf16", 3, 700, 5, 5, 40)])
def test_norm_without_eps(cuda_device, io, B, T, Hq, Hkv, dh):
    """eps = 0 is allowed: the places of a warp that have no row (heads that do not fill its rows)
    add nothing to dw, not 0 times the infinite root of nothing."""
    gen, q, k, w, pos = base.qk_inputs(io, B, T, Hq, Hkv, dh, 0, True, 81)
    q[0, 0, 0] = randn(gen, (dh,), io)                  # (a row of zeros has no norm without eps)
    dq, dk = randn(gen, q.shape, io), randn(gen, k.shape, io)
    rot = dh // 16 * 16
    d = [x.to(cuda_device) for x in (q, k, dq, dk, *w, pos)]
    got = rg.rglru_qk_norm_rope_bwd(*d, rot=rot, eps=0.0)
    for x, dy, wx, n in ((q, dq, w[0], "q"), (k, dk, w[1], "k")):
        check_norm_grads(got, x, dy, wx, pos, rot, io, 0.0, n)
        assert all(torch.isfinite(got[m]).all() for m in ("d" + n, "dw_" + n))


@pytest.mark.parametrize("io,fold", [("f32", 16), ("bf16", 64)])
def test_weight_gradients_of_many_rows(cuda_device, io, fold):
    """dw of millions of equal rows is off by no more than the few are (`fold` of them here) that a
    lane adds up before it folds them into an exact sum: a rounding each, beside the root's 4 u, the
    two products', the fold's and the store's."""
    B, T, dh = 4, 1 << 20, 8
    q = torch.ones(B, T, 1, dh, dtype=DT[io], device=cuda_device)
    dq = torch.full_like(q, 1 / 3)
    got = rg.rglru_qk_norm_rope_bwd(q, q.clone(), dq, dq.clone(), rot=0, eps=3.0)   # (root 1 / 2)
    ref = np.full(dh, B * T * float(dq[0, 0, 0, 0]) / 2)
    for n in ("dw_q", "dw_k"):
        close(got[n], ref, (8 + fold) * U * ref, n)


# ---------------------------------------------------------- what is not finite, who it reaches

@pytest.mark.parametrize("B", [1, 40])                  # split over clusters, and resident blocks
@pytest.mark.parametrize("dh,G", [(64, 1), (64, 2), (128, 1), (128, 2), (256, 2)])
def test_nan_key_in_every_column(cuda_device, dh, G, B):
    """A NaN in a key is the output and the log-sum of every query that sees it, whichever column
    of a tile it has (some go through another 2^x) and whether the mask cuts the tile or not."""
    T = 600
    gen = torch.Generator().manual_seed(91)
    q, k, v = (randn(gen, (B, T, h, dh), "bf16").to(cuda_device) for h in (2, 2 // G, 2 // G))
    out, lse = rg.rglru_local_attn_fwd(q, k, v)
    for key in (0, 1, 16, 17, 20, 33, 49, 127, 128, 160):
        k2 = k.clone()
        k2[B - 1, key, 0, 5] = float("nan")
        got, glse = rg.rglru_local_attn_fwd(q, k2, v)
        seen = torch.zeros(B, T, 2, dtype=torch.bool, device=cuda_device)
        seen[B - 1, key:, :G] = True                    # the query heads of key head 0
        assert torch.isnan(got[seen]).all() and torch.isnan(glse.transpose(1, 2)[seen]).all(), key
        assert torch.equal(got[~seen], out[~seen]), key
        assert torch.equal(glse.transpose(1, 2)[~seen], lse.transpose(1, 2)[~seen]), key


@pytest.mark.parametrize("dh", [64, 128, 256])
def test_nan_query_in_the_gradients(cuda_device, dh):
    """The gradients of the keys that a query with a NaN sees are NaN, whichever row it is."""
    T = 600
    gen = torch.Generator().manual_seed(92)
    q, k, v, dout = (randn(gen, (1, T, 1, dh), "bf16").to(cuda_device) for _ in range(4))
    for t in (256, 257, 272, 273, 276, 599):
        q2 = q.clone()
        q2[0, t, 0, 5] = float("nan")
        out, lse = rg.rglru_local_attn_fwd(q2, k, v)
        g = rg.rglru_local_attn_bwd(q2, k, v, out, lse, dout)
        assert torch.isnan(g["dq"][0, t]).all()
        assert torch.isnan(g["dk"][0, :t + 1]).all() and torch.isnan(g["dv"][0, :t + 1]).all(), t


@pytest.mark.parametrize("io,dh,B", [("bf16", 64, 1), ("bf16", 64, 40), ("bf16", 128, 1), ("bf16", 128, 40),
                                     ("bf16", 256, 1), ("bf16", 256, 40), ("bf16", 72, 1), ("f32", 64, 1)])
def test_scores_of_minus_infinity_weigh_nothing(cuda_device, io, dh, B):
    """A key whose score is -inf counts as one that is not seen, in every column; a query with no
    other key gets zeros and -inf."""
    T = 600
    gen = torch.Generator().manual_seed(93)
    q, k, v = (randn(gen, (B, T, 2, dh), io) for _ in range(3))
    q[..., 0] = 1.0
    k[0, :, 0, 0] = float("-inf")                       # all keys of a head
    k[0, 130:, 1, 0] = float("-inf")                    # the keys from 130 on
    q, k, v = (x.to(cuda_device) for x in (q, k, v))
    out, lse = rg.rglru_local_attn_fwd(q, k, v)
    assert torch.all(out[0, :, 0] == 0) and torch.all(torch.isneginf(lse[0, 0]))
    few = slice(130, T)                                 # those see keys 0 .. 129 of head 1
    kk = torch.where(torch.isinf(k), torch.zeros_like(k), k)
    ref, size, lref = whole_rows(f64(q[0, few, 1]), f64(kk[0, :130, 1]), f64(v[0, :130, 1]), dh ** -0.5)
    es = base.score_error(q[0, few, 1], kk[0, :130, 1], dh, dh ** -0.5)
    w = 2 * es + (T + 16) * 2 * U
    close(out[0, few, 1], ref, w * size + (UB * (size + np.abs(ref)) if io == "bf16" else 0), "out")
    close(lse[0, 1, few], lref, es + (T + 16) * 2 * U + 4 * U * np.abs(lref), "lse")


def whole_rows(q, k, v, scale):
    """Attention of every query over every key, in 64 bits."""
    z = scale * (q @ k.T)
    m = z.max(-1, keepdims=True)
    p = np.exp(z - m)
    l = p.sum(-1, keepdims=True)
    return p / l @ v, p / l @ np.abs(v), (np.log(l) + m)[:, 0]


@pytest.mark.parametrize("B", [1, 40])
@pytest.mark.parametrize("io,dh", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64)])
def test_scores_of_infinity_are_nan(cuda_device, io, dh, B):
    """A key whose score is +inf has no softmax: NaN for the queries that see it, in every column."""
    T = 600
    gen = torch.Generator().manual_seed(96)
    q, k, v = (randn(gen, (B, T, 2, dh), io) for _ in range(3))
    q[..., 0] = 1.0
    q, k, v = (x.to(cuda_device) for x in (q, k, v))
    out, lse = rg.rglru_local_attn_fwd(q, k, v)
    for key in (0, 17, 20, 160):
        k2 = k.clone()
        k2[B - 1, key, 1, 0] = float("inf")
        got, glse = rg.rglru_local_attn_fwd(q, k2, v)
        seen = torch.zeros(B, T, 2, dtype=torch.bool, device=cuda_device)
        seen[B - 1, key:, 1] = True
        assert torch.isnan(got[seen]).all() and torch.isnan(glse.transpose(1, 2)[seen]).all(), key
        assert torch.equal(got[~seen], out[~seen])


@pytest.mark.parametrize("io,dh,T,S", [("bf16", 64, 300, 173), ("bf16", 128, 150, 20), ("bf16", 256, 300, 173),
                                       ("bf16", 72, 100, 61), ("f32", 64, 100, 61), ("f32", 256, 70, 33)])
def test_queries_that_see_no_key_reach_no_gradient(cuda_device, io, dh, T, S):
    """With S < T the first T - S queries see no key: whatever they and their dout hold, their out
    is zero and the other rows' results are what they were."""
    gen = torch.Generator().manual_seed(94)
    q, dout = (randn(gen, (2, T, 4, dh), io).to(cuda_device) for _ in range(2))
    k, v = (randn(gen, (2, S, 2, dh), io).to(cuda_device) for _ in range(2))
    out, lse = rg.rglru_local_attn_fwd(q, k, v)
    g = rg.rglru_local_attn_bwd(q, k, v, out, lse, dout)
    q2, dout2 = q.clone(), dout.clone()
    q2[:, :T - S], dout2[:, :T - S] = float("nan"), float("inf")
    got, glse = rg.rglru_local_attn_fwd(q2, k, v)
    assert torch.equal(got, out) and torch.equal(glse, lse)
    assert torch.all(out[:, :T - S] == 0) and torch.all(torch.isneginf(lse[..., :T - S]))
    again = rg.rglru_local_attn_bwd(q2, k, v, out, lse, dout2)
    assert all(torch.equal(g[n], again[n]) for n in g)
    assert torch.all(g["dq"][:, :T - S] == 0)


# ---------------------------------------------------------------- one token over a cache

@pytest.mark.parametrize("io,dh,page,most", [("bf16", 8, 1 << 16, (1 << 15) - 1), ("bf16", 64, 1 << 16, (1 << 15) - 1),
                                             ("bf16", 8, 1, 2 ** 31 - 1), ("bf16", 64, 1, 2 ** 31 - 1)])
def test_paged_attn_decode_of_the_longest_tables(cuda_device, io, dh, page, most):
    """A table that names nearly 2^31 keys, or all of those, every page but the last one the same:
    equal scores, so that out is the mean of the values."""
    last = 2.0 ** 31 / page                             # (the last page weighs as much as the others)
    kc = torch.zeros(2, page, 1, dh, dtype=DT[io], device=cuda_device)
    vc = torch.ones_like(kc)
    vc[1] = last
    table = torch.zeros(1, most, dtype=torch.int32, device=cuda_device)
    table[0, -1] = 1
    q = torch.ones(1, 1, dh, dtype=DT[io], device=cuda_device)
    lens = torch.tensor([page * most], dtype=torch.int32, device=cuda_device)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    got = rg.rglru_paged_attn_decode(q, kc, vc, table, lens, dev_status=status)
    ref = np.full((1, 1, dh), (most - 1 + last) / most)
    # A block's sum of ones is a whole number below 2^24, exact; the last page adds equal numbers,
    # up to 65536 times 32768, powers of two; their sum and the join's of up to 1024 parts round.
    close(got, ref, (1100 * 2 * U + UB) * ref, "out")
    assert int(status) == 0


@pytest.mark.parametrize("io,dh", [("bf16", 128), ("f32", 64), ("bf16", 72)])
@pytest.mark.parametrize("window,sinks", [(20, 3), (20, 0), (31, 40), (5, 2)])
def test_paged_attn_decode_past_its_table(cuda_device, io, dh, window, sinks):
    """A length past what its table names is reported, and the keys past it are hidden: the window
    stays where the length puts it."""
    page, most = 8, 4
    gen = torch.Generator().manual_seed(95)
    lens = [45, 33, 32, 70, 2 ** 31 - 1, 52, 20]
    B, cap = len(lens), page * most
    table = torch.randperm(B * most, generator=gen).view(B, most).to(torch.int32)
    q = randn(gen, (B, 4, dh), io)
    kc, vc = (randn(gen, (B * most, page, 2, dh), io) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    d = [x.to(cuda_device) for x in (q, kc, vc, table, torch.tensor(lens, dtype=torch.int32))]
    got = rg.rglru_paged_attn_decode(*d, window=window, sinks=sinks, dev_status=status)
    assert int(status) == 1
    for b, n in enumerate(lens):
        keys = [j for j in range(min(n, cap)) if j > n - 1 - window or j < sinks]
        if not keys:
            assert torch.all(got[b] == 0)
            continue
        at = [(int(table[b, j // page]), j % page) for j in keys]
        k, v = (np.stack([f64(c[p, s]) for p, s in at])[None] for c in (kc, vc))
        ref, size = orc.paged_decode(f64(q[b:b + 1]), k, v, np.zeros((1, 1), int), [len(keys)], 0, 0, dh ** -0.5)
        w = 2 * base.score_error(q, torch.tensor(k), dh, dh ** -0.5) + (cap + 16) * 2 * U
        close(got[b:b + 1], ref, w * size + (UB * (size + np.abs(ref)) if io == "bf16" else 0), b)


# ------------------------------------------------------- several units of work a block or warp

MANY = [  # 370 units of work and more over the resident blocks of the forward
    ("bf16", 4, 700, 700, 32, 16, 64, 200, 2, [700, 0, 513, 90], "slice"),
    ("bf16", 4, 1000, 1000, 36, 12, 64, 0, 0, [1000, 300, 0, 640], "dense"),
    ("bf16", 3, 900, 900, 40, 20, 128, 0, 0, None, "heads"),
    ("bf16", 4, 600, 900, 30, 10, 128, 250, 140, None, "slice"),
    ("bf16", 4, 600, 600, 20, 2, 256, 300, 3, [600, 431, 1, 600], "slice"),
]


@pytest.mark.parametrize("case", MANY, ids=str)
def test_local_attn_of_many_units(cuda_device, case):
    base.test_local_attn_fwd(cuda_device, case)


@pytest.mark.parametrize("case", MANY[::2], ids=str)
def test_local_attn_bwd_of_many_blocks(cuda_device, case):
    base.test_local_attn_bwd(cuda_device, case)


@pytest.mark.parametrize("case", [("bf16", 8, 1250, 10, 1, 64, 64, "slice", 0, True),
                                  ("f32", 8, 1250, 3, 2, 128, 64, "heads", 9000, True),
                                  ("bf16", 5, 1700, 4, 1, 256, 128, "slice", 70, False)], ids=str)
def test_norms_of_many_tokens(cuda_device, case):
    """More tokens than warps: each takes several, with all of a token's heads."""
    base.test_qk_norm_rope_fwd(cuda_device, case)
    base.test_qk_norm_rope_bwd(cuda_device, case)


@pytest.mark.parametrize("io,Hq,Hkv,dh,window,sinks", [("bf16", 10, 1, 256, 100, 4), ("bf16", 4, 2, 64, 0, 0),
                                                       ("f32", 4, 2, 64, 50, 1)])
def test_paged_attn_decode_of_many_sequences(cuda_device, io, Hq, Hkv, dh, window, sinks):
    lens = [(b * 37) % 331 for b in range(200)]
    base.test_paged_attn_decode(cuda_device, (io, Hq, Hkv, dh, 16, lens, window, sinks, 22))


# --------------------------------------------------------------- calls that are allowed, and odd

@pytest.mark.parametrize("io,dh", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64)])
def test_lengths_out_of_range_are_clamped(cuda_device, io, dh):
    gen = torch.Generator().manual_seed(97)
    q, k, v, dout = (randn(gen, (4, 150, h, dh), io).to(cuda_device) for h in (4, 2, 2, 4))
    got = []
    for lens in ([-3, 2 ** 31 - 1, 0, 150], [0, 150, 0, 150]):
        n = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
        out, lse = rg.rglru_local_attn_fwd(q, k, v, window=40, sinks=1, lens=n)
        got.append([out, lse, *rg.rglru_local_attn_bwd(q, k, v, out, lse, dout, window=40, sinks=1, lens=n).values()])
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("io,Hq,Hkv,dh,window,sinks", [("bf16", 16, 4, 128, 0, 0), ("bf16", 10, 1, 256, 300, 4),
                                                       ("f32", 4, 2, 64, 0, 0)])
def test_paged_attn_decode_under_a_wide_table(cuda_device, io, Hq, Hkv, dh, window, sinks):
    """A table for far more keys than the sequences have, its other entries anything; and lengths
    below zero."""
    case = (io, Hq, Hkv, dh, 16, [700, 0, 33, 512], window, sinks, 44)
    q, kc, vc, table, lens = base.decode_inputs(case, 24)
    wide = torch.randint(-2 ** 31, 2 ** 31 - 1, (4, 8192), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    wide[:, :44] = table
    lens[1] = -7
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    d = [x.to(cuda_device) for x in (q, kc, vc, wide, lens)]
    got = rg.rglru_paged_attn_decode(*d, window=window, sinks=sinks, dev_status=status)
    assert int(status) == 0 and torch.all(got[1] == 0)
    scale = dh ** -0.5
    ref, size = orc.paged_decode(f64(q), f64(kc), f64(vc), table.numpy(), lens.tolist(), window, sinks, scale)
    w = 2 * base.score_error(q, kc, dh, scale) + (700 + 16) * 2 * U
    close(got, ref, w * size + (UB * (size + np.abs(ref)) if io == "bf16" else 0), "out")


@pytest.mark.parametrize("B,T,S,dh", [(2, 900, 900, 64), (1, 30, 3000, 128), (2, 700, 700, 256)])
def test_two_calls_at_once(cuda_device, B, T, S, dh):
    """Resident blocks, or clusters, of two calls on two streams share the GPU: each gets its bits."""
    gen = torch.Generator().manual_seed(98)
    sets = [[randn(gen, (B, n, h, dh), "bf16").to(cuda_device) for n, h in ((T, 20), (S, 2), (S, 2), (T, 20))]
            for _ in range(2)]

    def calls(x, stream=None):
        q, k, v, dout = x
        out, lse = rg.rglru_local_attn_fwd(q, k, v, window=S // 2, sinks=2, stream=stream)
        g = rg.rglru_local_attn_bwd(q, k, v, out, lse, dout, window=S // 2, sinks=2, stream=stream)
        return [out, lse, *g.values()]

    ref = [calls(x) for x in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[calls(x, s) for x, s in zip(sets, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(a, b) for x, y in zip(pair, ref) for a, b in zip(x, y))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dh", range(8, 257, 8))
def test_every_width(cuda_device, io, dh):
    """Norm, rotation, attention, their backwards and the decode, for every width of a head."""
    norm = (io, 2, 7, 3, 1, dh, dh // 16 * 16, "slice", 40, True)
    base.test_qk_norm_rope_fwd(cuda_device, norm)
    base.test_qk_norm_rope_bwd(cuda_device, norm)
    attn = (io, 2, 70, 75, 2, 1, dh, 30, 2, None, "slice")
    base.test_local_attn_fwd(cuda_device, attn)
    base.test_local_attn_bwd(cuda_device, attn)
    base.test_paged_attn_decode(cuda_device, (io, 3, 1, dh, 5, [40, 300], 50, 1, 60))
