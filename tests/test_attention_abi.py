"""CPU checks of the local attention entry points: bad arguments are refused
before any launch, and the host's plan of a call covers it."""
import ctypes

import pytest
import torch

from gated_linear_recurrence_rglru_b200.attention import LIB, Strides
import gated_linear_recurrence_rglru_b200 as rg

FAKE = 1 << 24  # 16-byte aligned stand-in, spaced by the calls; never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


def at(i):
    return FAKE * (i + 1)


def strides(*s):
    return ctypes.byref(Strides(*s))


def qk_fwd(**o):
    a = dict(q=at(0), qs=None, k=at(1), ks=None, w_q=at(2), w_k=at(3), pos=at(4), q_out=at(5),
             k_out=at(6), B=2, T=3, Hq=4, Hkv=2, dh=64, rot=64, base=1e4, eps=1e-6, io=1)
    a.update(o)
    return LIB.rglru_qk_norm_rope_fwd(*a.values(), None)


def qk_append(**o):
    a = dict(q=at(0), qs=None, k=at(1), ks=None, v=at(2), vs=None, w_q=None, w_k=None, pos=at(3),
             q_out=at(4), k_cache=at(5), v_cache=at(6), table=at(7), pages=4, page=16, most=2, B=2,
             T=3, Hq=4, Hkv=2, dh=64, rot=64, base=1e4, eps=1e-6, io=1, status=None)
    a.update(o)
    return LIB.rglru_qk_norm_rope_append(*a.values(), None)


def qk_bwd(**o):
    a = dict(q=at(0), qs=None, k=at(1), ks=None, w_q=None, w_k=None, pos=None, dqo=at(2),
             dko=at(3), dq=at(4), dk=at(5), dwq=at(6), dwk=at(7), B=2, T=3, Hq=4, Hkv=2, dh=64,
             rot=64, base=1e4, eps=1e-6, io=1, ws=at(8), n=1 << 22)
    a.update(o)
    return LIB.rglru_qk_norm_rope_bwd(*a.values(), None)


def attn_fwd(**o):
    a = dict(q=at(0), qs=None, k=at(1), ks=None, v=at(2), vs=None, lens=None, out=at(3), lse=at(4),
             B=2, T=8, S=8, Hq=4, Hkv=2, dh=64, window=0, sinks=0, scale=0.125, io=1, status=None)
    a.update(o)
    return LIB.rglru_local_attn_fwd(*a.values(), None)


def attn_bwd(**o):
    a = dict(q=at(0), qs=None, k=at(1), ks=None, v=at(2), vs=None, out=at(3), lse=at(4),
             dout=at(5), lens=None, dq=at(6), dk=at(7), dv=at(8), B=2, T=8, S=8, Hq=4, Hkv=2,
             dh=64, window=0, sinks=0, scale=0.125, io=1, ws=at(9), n=1 << 23, status=None)
    a.update(o)
    return LIB.rglru_local_attn_bwd(*a.values(), None)


def decode(**o):
    a = dict(q=at(0), kc=at(1), vc=at(2), table=at(3), lens=at(4), out=at(5), pages=8, page=16,
             most=4, B=2, Hq=4, Hkv=2, dh=64, window=0, sinks=0, scale=0.125, io=1, ws=at(6),
             n=1 << 22, status=None)
    a.update(o)
    return LIB.rglru_paged_attn_decode(*a.values(), None)


HEADS = [(dict(B=0), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=-1), INVALID), (dict(dh=0), INVALID),
         (dict(dh=60), INVALID), (dict(dh=264), UNSUPPORTED), (dict(io=2), INVALID),
         (dict(B=1 << 20, Hkv=1, Hq=1), UNSUPPORTED)]
NORMS = [(dict(T=0), INVALID), (dict(rot=8), INVALID), (dict(rot=-16), INVALID),
         (dict(rot=80), INVALID), (dict(base=0.5), INVALID), (dict(base=float("nan")), INVALID),
         (dict(base=float("inf")), INVALID), (dict(eps=-1e-6), INVALID),
         (dict(eps=float("nan")), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
         (dict(q=at(0) + 8), INVALID), (dict(pos=at(4) + 4), INVALID), (dict(w_q=at(2) + 2), INVALID),
         (dict(qs=strides(768, 260, 64)), INVALID),      # a stride that is no whole 16 bytes
         (dict(qs=strides(768, 0, 64)), INVALID),        # a broadcast dimension
         (dict(qs=strides(768, 256, -64)), INVALID),
         (dict(ks=strides(1 << 40, 256, 64)), INVALID)]
ATTN = [(dict(T=0), INVALID), (dict(S=0), INVALID), (dict(Hq=3), INVALID), (dict(window=-1), INVALID),
        (dict(sinks=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
        (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
        (dict(lens=at(20), S=9), INVALID), (dict(lens=at(20) + 4), INVALID), (dict(v=None), INVALID),
        (dict(out=None), INVALID), (dict(vs=strides(1024, 100, 64)), INVALID),
        (dict(out=at(0)), INVALID), (dict(out=at(2) + 16), INVALID),
        (dict(T=3 << 20, S=3 << 20, B=1), UNSUPPORTED)]


@pytest.mark.parametrize("over,code", HEADS + NORMS + [
    (dict(q_out=at(0)), INVALID), (dict(k_out=at(5)), INVALID), (dict(k_out=None), INVALID)])
def test_qk_fwd_refuses(over, code):
    assert qk_fwd(**over) == code


@pytest.mark.parametrize("over,code", HEADS + NORMS + [
    (dict(v=None), INVALID), (dict(pos=None), INVALID), (dict(table=None), INVALID),
    (dict(pages=0), INVALID), (dict(page=0), INVALID), (dict(most=0), INVALID),
    (dict(v_cache=at(5)), INVALID), (dict(v_cache=at(2)), INVALID), (dict(q_out=at(2)), INVALID),
    (dict(pages=1 << 30, page=1 << 30), UNSUPPORTED), (dict(status=at(9) + 4), INVALID)])
def test_qk_append_refuses(over, code):
    assert qk_append(**over) == code


@pytest.mark.parametrize("over,code", HEADS + NORMS + [
    (dict(dqo=None), INVALID), (dict(dq=at(0)), INVALID), (dict(dq=at(2)), INVALID),
    (dict(dwk=at(6)), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=at(8) + 8), WORKSPACE),
    (dict(n=16), WORKSPACE), (dict(ws=at(4)), INVALID)])
def test_qk_bwd_refuses(over, code):
    assert qk_bwd(**over) == code


@pytest.mark.parametrize("over,code", HEADS + ATTN + [(dict(lse=at(3)), INVALID)])
def test_attn_fwd_refuses(over, code):
    assert attn_fwd(**over) == code


@pytest.mark.parametrize("over,code", HEADS + [c for c in ATTN if "out" not in c[0]] + [
    (dict(lse=None), INVALID), (dict(dq=at(5)), INVALID), (dict(dk=at(8)), INVALID),
    (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE), (dict(ws=at(7)), INVALID)])
def test_attn_bwd_refuses(over, code):
    assert attn_bwd(**over) == code


@pytest.mark.parametrize("over,code", HEADS + [
    (dict(Hq=3), INVALID), (dict(pages=0), INVALID), (dict(page=0), INVALID), (dict(most=0), INVALID),
    (dict(window=-1), INVALID), (dict(sinks=-2), INVALID), (dict(scale=0.0), INVALID),
    (dict(lens=None), INVALID), (dict(out=at(0)), INVALID), (dict(out=at(1) + 64), INVALID),
    (dict(ws=None), WORKSPACE), (dict(n=8), WORKSPACE), (dict(ws=at(5)), INVALID),
    (dict(page=1 << 20, most=1 << 20), UNSUPPORTED)])
def test_decode_refuses(over, code):
    assert decode(**over) == code


def test_workspace_sizes_of_bad_sizes_are_zero():
    assert LIB.rglru_local_attn_bwd_workspace_bytes(2, 8, 8, 3, 2, 64, 0, 0, 1) == 0
    assert LIB.rglru_local_attn_bwd_workspace_bytes(2, 8, 8, 4, 2, 64, 0, 0, 1) > 0
    assert LIB.rglru_qk_norm_rope_bwd_workspace_bytes(2, 8, 4, 2, 60, 1) == 0
    assert LIB.rglru_qk_norm_rope_bwd_workspace_bytes(2, 8, 4, 2, 64, 1) > 0
    assert LIB.rglru_paged_attn_decode_workspace_bytes(2, 4, 3, 64, 16, 4, 0, 0, 1) == 0
    # few sequences with a long cache are split: room for the parts
    assert LIB.rglru_paged_attn_decode_workspace_bytes(1, 4, 1, 64, 16, 4096, 0, 0, 1) > 4 * 64 * 4


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 4, 2, 64)
    for call in (lambda: rg.rglru_qk_norm_rope_fwd(x, x), lambda: rg.rglru_local_attn_fwd(x, x, x),
                 lambda: rg.rglru_paged_attn_decode(x[0], x, x, torch.zeros(1, 1), torch.zeros(1))):
        with pytest.raises(TypeError):
            call()
