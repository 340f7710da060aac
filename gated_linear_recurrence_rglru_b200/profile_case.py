"""Run a few calls of one workload through the library, for profiler captures.

    python -m gated_linear_recurrence_rglru_b200.profile_case long_context:16384 3
    python -m gated_linear_recurrence_rglru_b200.profile_case decode_batch 4
    python -m gated_linear_recurrence_rglru_b200.profile_case local_attention:2048 2

A forward workload (optionally cut to T tokens with `name:T`) runs `calls`
forwards on rotating copies of x, so that consecutive launches do not find
their input in L2; `decode_batch` runs `calls` decode steps. The inputs are the
workload's seeded synthetic recipe. `local_attention` runs `calls` times the layer's
other mixing at griffin2b's width (D = 2560 as 10 query heads on one 256-wide key
head, window 1024): a training step of 4 rows (norm and rotation, attention, both
backwards), the rows' keys and values into a paged cache, and a decode step over it.
Exits non-zero if a call reports an error.
A profiler then selects launches by kernel name and index, e.g.
`ncu -k regex:fwd_tc -s 1 -c 1 ...`.
"""
from __future__ import annotations

import argparse
import sys

import torch

from . import _abi, attention
from .workloads import WORKLOADS, generate

WEIGHTS = ("conv_w", "W_a", "b_a", "W_x", "b_x", "Lambda")


def _device_inputs(wl, dev):
    t = generate(wl)
    return {k: (v.to(dev) if isinstance(v, torch.Tensor) else v) for k, v in t.items()}


def run_forward(wl, calls: int, dev) -> None:
    g = _device_inputs(wl, dev)
    w = [g[k] for k in WEIGHTS]
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    xs = [g["x"]] + [g["x"].clone() for _ in range(2)]
    y = torch.empty_like(g["x"])
    for i in range(calls):
        _abi.rglru_fwd(xs[i % len(xs)], *w, h0=g["h0"], dev_status=status, y=y)
    torch.cuda.synchronize(dev)
    if int(status.item()) != 0:
        raise SystemExit(f"forward reported status word {int(status.item()):#x}")


def run_decode(wl, calls: int, dev) -> None:
    g = _device_inputs(wl.with_shape(decode_steps=calls), dev)
    w = [g[k] for k in WEIGHTS]
    h, ring = g["h"].clone(), g["conv_state"].clone()
    for s in range(calls):
        _abi.rglru_decode_step(g["x_steps"][s], ring, s, h, *w)
    torch.cuda.synchronize(dev)


def run_local_attention(T: int, calls: int, dev) -> None:
    B, Hq, Hkv, dh, window, page = 4, 10, 1, 256, 1024, 16
    gen = torch.Generator(device=dev).manual_seed(0)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev).bfloat16()

    status = torch.zeros(1, dtype=torch.int32, device=dev)
    pages = -(-T // page)
    table = torch.arange(B * pages, dtype=torch.int32, device=dev).view(B, pages)
    positions = torch.arange(T, dtype=torch.int32, device=dev).expand(B, T).contiguous()
    lens = torch.full((B,), T, dtype=torch.int32, device=dev)
    k_cache, v_cache = (randn(B * pages, page, Hkv, dh) for _ in range(2))
    for _ in range(calls):
        q, k, v = randn(B, T, Hq + 2 * Hkv, dh).split([Hq, Hkv, Hkv], 2)
        qn, kn = attention.rglru_qk_norm_rope_fwd(q, k, rot=dh // 2)
        out, lse = attention.rglru_local_attn_fwd(qn, kn, v, window=window, dev_status=status)
        g = attention.rglru_local_attn_bwd(qn, kn, v, out, lse, randn(B, T, Hq, dh), window=window,
                                           dev_status=status)
        attention.rglru_qk_norm_rope_bwd(q, k, g["dq"], g["dk"], rot=dh // 2)
        qa = attention.rglru_qk_norm_rope_append(q, k, v, k_cache, v_cache, table, positions,
                                                 rot=dh // 2, dev_status=status)
        attention.rglru_paged_attn_decode(qa[:, -1].contiguous(), k_cache, v_cache, table, lens,
                                          window=window, dev_status=status)
    torch.cuda.synchronize(dev)
    if int(status.item()) != 0:
        raise SystemExit(f"attention reported status word {int(status.item()):#x}")


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("case", help="workload name or local_attention, optionally name:T for T tokens")
    ap.add_argument("calls", type=int, nargs="?", default=3)
    args = ap.parse_args(argv)
    name, _, T = args.case.partition(":")
    if name not in WORKLOADS and name != "local_attention":
        ap.error(f"unknown workload {name!r} (one of {', '.join(WORKLOADS)}, local_attention)")
    if not torch.cuda.is_available():
        raise SystemExit("profile_case needs a CUDA device")
    dev = torch.device("cuda:0")
    if name == "local_attention":
        run_local_attention(int(T or 2048), args.calls, dev)
        print("ok", args.case, args.calls)
        return 0
    wl = WORKLOADS[name]
    if wl.decode_steps > 0:
        run_decode(wl, args.calls, dev)
    else:
        run_forward(wl.with_shape(T=int(T)) if T else wl, args.calls, dev)
    print("ok", args.case, args.calls)
    return 0


if __name__ == "__main__":
    sys.exit(main())
