"""CPU checks of the local attention entry points: strides whose products with a size pass 64
bits are refused, not taken for the short span that is left of them."""
import pytest

from test_attention_abi import INVALID, WORKSPACE, attn_bwd, attn_fwd, qk_append, qk_bwd, qk_fwd, strides

N = 1 << 26          # (N + 1 rows) x 2^38 elements: 2^64, which is 0 in 64 bits
FAR = 1 << 38        # the largest stride that is accepted


def spaced(*names):
    """Stand-ins far enough apart for the sizes here; never dereferenced."""
    return {n: (i + 1) << 44 for i, n in enumerate(names)}


QK = spaced("q", "k", "w_q", "w_k", "pos", "q_out", "k_out")
APPEND = spaced("q", "k", "v", "pos", "q_out", "k_cache", "v_cache", "table")
QK_BWD = spaced("q", "k", "dqo", "dko", "dq", "dk", "dwq", "dwk", "ws")
ATTN = spaced("q", "k", "v", "out", "lse")
ATTN_BWD = spaced("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "ws")
TOKENS = dict(B=1, T=N + 1, Hq=1, Hkv=1, dh=8, qs=strides(8, FAR, 8))
BATCH = dict(B=(1 << 15) + 1, T=1, Hq=1, Hkv=1, dh=8, qs=strides(FAR, 8, 8))      # 2^53: no device has it
HEADS = dict(B=1, T=1, Hq=N + 1, Hkv=1, dh=8, qs=strides(8, 8, FAR))
KEYS = dict(B=1, T=N + 1, Hq=1, Hkv=1, dh=8, ks=strides(8, FAR, 8))


@pytest.mark.parametrize("over", [TOKENS, BATCH, HEADS, KEYS])
@pytest.mark.parametrize("call,at", [(qk_fwd, QK), (qk_append, APPEND), (qk_bwd, QK_BWD)])
def test_norms_refuse_spans_past_64_bits(call, at, over):
    more = dict(n=1 << 40) if call is qk_bwd else {}
    assert call(**{**at, **over, **more, "rot": 0}) == INVALID


@pytest.mark.parametrize("call,at", [(attn_fwd, ATTN), (attn_bwd, ATTN_BWD)])
@pytest.mark.parametrize("over", [{**HEADS, "S": 1}, {**BATCH, "S": 1},
                                  dict(B=1, T=1, S=(1 << 20) + 1, Hq=1, Hkv=1, dh=8, ks=strides(8, FAR, 8)),
                                  dict(B=1, T=1, S=(1 << 20) + 1, Hq=1, Hkv=1, dh=8, vs=strides(8, FAR, 8))])
def test_attention_refuses_spans_past_any_device(call, at, over):
    more = dict(n=1 << 40) if call is attn_bwd else {}
    assert call(**{**at, **over, **more}) == INVALID


@pytest.mark.parametrize("over", [dict(qs=strides(FAR, 256, 64)), dict(B=1, T=2, S=2, qs=strides(8, FAR, 64)),
                                  dict(B=1, T=2, S=2, Hq=2, Hkv=2, vs=strides(8, 64, FAR))])
def test_the_largest_strides_are_taken(over):
    """A single step of 2^38 elements passes the check of the strides: the next one, of the
    workspace's size, is what refuses."""
    assert attn_bwd(**{**ATTN_BWD, **over, "n": 16}) == WORKSPACE
    assert attn_bwd(**{**ATTN_BWD, "qs": strides(FAR + 8, FAR + 8, FAR + 8), "n": 16}) == INVALID
