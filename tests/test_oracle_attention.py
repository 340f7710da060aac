"""Pins of the float64 attention oracle (oracle/attention_oracle.py), on the CPU: closed
forms, torch's own float64 operators, and central differences."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as orc

RNG = np.random.default_rng(7)


def test_rotation_keeps_norms_and_differences():
    x, y = RNG.standard_normal((2, 1, 1, 1, 32))
    for a, b in ((3, 10), (100003, 100010)):
        xa = orc.rotation(x, np.array([[a]]), 32, 10000.0)
        yb = orc.rotation(y, np.array([[b]]), 32, 10000.0)
        dot = float((xa * yb).sum())
        ref = float((orc.rotation(x, np.array([[0]]), 32, 10000.0)
                     * orc.rotation(y, np.array([[7]]), 32, 10000.0)).sum())
        assert abs(dot - ref) < 1e-9          # only the difference of positions counts
        assert abs(np.linalg.norm(xa) - np.linalg.norm(x)) < 1e-12
    back = orc.rotation(orc.rotation(x, np.array([[5]]), 16, 100.0), np.array([[5]]), 16, 100.0, True)
    assert np.allclose(back, x, atol=1e-14)


def test_norm_matches_torch():
    x, w = RNG.standard_normal((2, 3, 4, 24)), RNG.standard_normal(24)
    y = orc.qk_norm_rope(x, w, np.zeros((2, 3)), 16, 10000.0, 1e-6)
    ref = torch.nn.functional.rms_norm(torch.tensor(x), (24,), torch.tensor(w), 1e-6).numpy()
    assert np.allclose(y, ref, atol=1e-12)    # position 0 turns nothing


def test_norm_rope_backward_by_differences():
    x, w, dy = RNG.standard_normal((2, 2, 2, 16)), RNG.standard_normal(16), RNG.standard_normal((2, 2, 2, 16))
    pos = np.array([[0, 5], [9, -3]])
    f = lambda x, w: float((orc.qk_norm_rope(x, w, pos, 16, 50.0, 1e-3) * dy).sum())  # noqa: E731
    dx, dw = orc.qk_norm_rope_bwd(x, w, dy, pos, 16, 50.0, 1e-3)
    e = 1e-6
    for i in ((0, 0, 0, 0), (1, 1, 1, 15), (0, 1, 0, 7)):
        d = np.zeros_like(x)
        d[i] = e
        assert abs((f(x + d, w) - f(x - d, w)) / (2 * e) - dx[i]) < 1e-7
    for i in (0, 9):
        d = np.zeros_like(w)
        d[i] = e
        assert abs((f(x, w + d) - f(x, w - d)) / (2 * e) - dw[i]) < 1e-7


@pytest.mark.parametrize("T,S,window,sinks", [(5, 5, 0, 0), (6, 9, 3, 1), (7, 4, 2, 0), (4, 4, 1, 2)])
def test_local_attn_matches_torch(T, S, window, sinks):
    B, Hq, Hkv, dh = 2, 4, 2, 8
    q, k, v = (RNG.standard_normal(s) for s in ((B, T, Hq, dh), (B, S, Hkv, dh), (B, S, Hkv, dh)))
    out, lse, _ = orc.local_attn(q, k, v, window, sinks, 0.3)
    ok = np.zeros((T, S), dtype=bool)         # the mask, position by position
    for t in range(T):
        p = t + S - T
        for j in range(S):
            ok[t, j] = j <= p and (window == 0 or p - j < window or j < sinks)
    tq, tk, tv = (torch.tensor(x).transpose(1, 2) for x in (q, k, v))
    z = tq @ tk.repeat_interleave(2, 1).transpose(-1, -2) * 0.3
    z = z.masked_fill(~torch.tensor(ok), float("-inf"))
    ref = torch.nan_to_num(torch.softmax(z, -1)) @ tv.repeat_interleave(2, 1)
    assert np.allclose(out, ref.transpose(1, 2).numpy(), atol=1e-12)
    assert np.allclose(lse, torch.logsumexp(z, -1).numpy(), atol=1e-12)
    empty = ~ok.any(-1)
    assert np.all(out[:, empty] == 0) and np.all(np.isneginf(lse[:, :, empty]))


def test_local_attn_backward_by_differences():
    B, T, S, Hq, Hkv, dh, window, sinks = 1, 5, 7, 4, 2, 4, 3, 1
    q, k, v = (RNG.standard_normal(s) for s in ((B, T, Hq, dh), (B, S, Hkv, dh), (B, S, Hkv, dh)))
    dout = RNG.standard_normal(q.shape)
    out, _, _ = orc.local_attn(q, k, v, window, sinks, 0.5)
    g, _, _ = orc.local_attn_bwd(q, k, v, out, dout, window, sinks, 0.5)
    f = lambda q, k, v: float((orc.local_attn(q, k, v, window, sinks, 0.5)[0] * dout).sum())  # noqa: E731
    e = 1e-6
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        for i in np.ndindex(x.shape):
            d = np.zeros_like(x)
            d[i] = e
            a = [y + d if y is x else y for y in (q, k, v)]
            b = [y - d if y is x else y for y in (q, k, v)]
            assert abs((f(*a) - f(*b)) / (2 * e) - g[name][i]) < 1e-7, (name, i)


def test_ragged_rows_equal_single_rows():
    lens = [4, 0, 6]
    q, k, v = RNG.standard_normal((3, 3, 6, 2, 8))
    out, lse, _ = orc.local_attn(q, k, v, 3, 1, 0.4, lens)
    for b, n in enumerate(lens):
        if n:
            o, l, _ = orc.local_attn(q[b:b + 1, :n], k[b:b + 1, :n], v[b:b + 1, :n], 3, 1, 0.4)
            assert np.array_equal(out[b:b + 1, :n], o) and np.array_equal(lse[b:b + 1, :, :n], l)
        assert np.all(np.isnan(out[b, n:]))


def test_paged_decode_is_the_last_row_of_attention():
    B, Hq, Hkv, dh, page = 3, 4, 2, 8, 4
    lens, window, sinks = [1, 9, 14], 5, 2
    table = RNG.permutation(B * 4).reshape(B, 4)
    kc, vc = RNG.standard_normal((2, B * 4, page, Hkv, dh))
    q = RNG.standard_normal((B, Hq, dh))
    out, _ = orc.paged_decode(q, kc, vc, table, lens, window, sinks, 0.4)
    for b, n in enumerate(lens):
        k = np.stack([kc[table[b, j // page], j % page] for j in range(n)])[None]
        v = np.stack([vc[table[b, j // page], j % page] for j in range(n)])[None]
        o, _, _ = orc.local_attn(q[b:b + 1, None], k, v, window, sinks, 0.4)
        assert np.allclose(out[b], o[0, 0], atol=1e-13)
