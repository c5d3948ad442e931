#!/usr/bin/env python
"""Run one SDPA operation repeatedly on one synthetic case, for profilers (ncu) and quick
timing.  Every launch goes through the C ABI exactly as in normal use.

  python bench_profile.py --op fwd|bwd|step \\
      --B 2 --Hq 32 --Hkv 8 --L 4096 --D 128 --dtype bf16 --causal --iters 4 \\
      [--mask padding|additive]

--L is Lq (and Lkv unless --Lkv is given).  --mask padding passes a boolean key-padding
mask [B, 1, 1, Lkv] hiding the last 10% of the keys; --mask additive passes one N(0, 1)
[Lq, Lkv] mask in the element type, shared by every batch and head (seed 6).  The cache
operations work on sequences of --Lkv tokens in pages of --page tokens, in random order, and
on the last --L rows of each; rotary turns q and k of --L rows by positions that end at --Lkv.
Prints the mean CUDA-event time per call (after one warm-up call).
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from scaled_dot_product_flash_gb300 import _lib, api  # noqa: E402
from scaled_dot_product_flash_gb300.inputs import Shape, draw  # noqa: E402


def timed(once, iters):
    """Mean CUDA-event time of a call, after one warm-up call."""
    once()
    api.poll_status()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(iters):
        once()
    e1.record()
    api.poll_status()
    return e0.elapsed_time(e1) / iters


def serving_op(a):
    """(call, bytes it has to move) of one rotary or cache operation on its synthetic case."""
    shape = Shape(a.B, a.Hq, a.Hkv, a.L, a.L, a.D)
    n = a.Lkv or a.L
    q, k, v, _ = (t.cuda() for t in draw(shape, 3, a.dtype))
    es, row = q.element_size(), a.B * a.Hkv * a.D
    if a.op == "rotary":
        inv = (10000.0 ** (-torch.arange(a.D // 2, dtype=torch.float64) * 2 / a.D)).float().cuda()
        positions = torch.arange(n - a.L, n, device="cuda")
        outs = (torch.empty_like(q), torch.empty_like(k))
        return (lambda: api.rotary(q, k, positions, inv, q_out=outs[0], k_out=outs[1]),
                2 * es * (q.numel() + k.numel()))
    per = -(-n // a.page)
    pages = torch.randperm(a.B * per, generator=torch.Generator().manual_seed(7))
    pages = pages.to(torch.int32).view(a.B, per).cuda()
    lens = torch.full((a.B,), n, dtype=torch.int32, device="cuda")
    cache = api.cache_empty(a.B * per, a.Hkv, a.page, a.D, q.dtype)
    gen = torch.Generator(device="cuda").manual_seed(8)
    for at in range(0, n, 4096):  # fill it
        rows = min(4096, n - at)
        new = [torch.randn(a.B, a.Hkv, rows, a.D, generator=gen, device="cuda").to(q.dtype)
               for _ in range(2)]
        api.cache_write(cache, *new, pages, torch.full_like(lens, at + rows))
    if a.op == "cache_write":
        return lambda: api.cache_write(cache, k, v, pages, lens), row * a.L * (2 * es + 1.25)
    if a.op == "cache_read":
        outs = (torch.empty_like(k), torch.empty_like(v))
        return (lambda: api.cache_read(cache, pages, lens, a.L, k=outs[0], v=outs[1]),
                row * a.L * (2 * es + 1.25))
    out = torch.empty_like(q)
    return (lambda: api.cache_attention(q, cache, pages, lens, out=out),
            row * n * 1.25 + 2 * es * q.numel())


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--op", choices=["fwd", "bwd", "step", "rotary", "cache_write",
                                     "cache_read", "cache_attn"], default="fwd")
    ap.add_argument("--B", type=int, default=2)
    ap.add_argument("--Hq", type=int, default=32)
    ap.add_argument("--Hkv", type=int, default=8)
    ap.add_argument("--L", type=int, default=4096)
    ap.add_argument("--Lkv", type=int, default=None)
    ap.add_argument("--D", type=int, default=128)
    ap.add_argument("--dtype", default="bf16", choices=["f32", "f16", "bf16"])
    ap.add_argument("--causal", action="store_true")
    ap.add_argument("--path", default="auto", choices=["auto", "tensor", "simt", "vector"])
    ap.add_argument("--iters", type=int, default=4)
    ap.add_argument("--mask", default="none", choices=["none", "padding", "additive"])
    ap.add_argument("--page", type=int, default=64)
    a = ap.parse_args()
    if a.op not in ("fwd", "bwd", "step"):
        once, nbytes = serving_op(a)
        ms = timed(once, a.iters)
        print(f"{a.op}: {ms:.4f} ms per call, {nbytes / ms / 1e6:.1f} GB/s")
        return
    shape = Shape(a.B, a.Hq, a.Hkv, a.L, a.Lkv or a.L, a.D)
    q, k, v, do = (t.cuda() for t in draw(shape, 3, a.dtype))
    scale = 1.0 / math.sqrt(a.D)
    Lkv = a.Lkv or a.L
    mask = None
    if a.mask == "padding":
        mask = torch.ones(a.B, 1, 1, Lkv, dtype=torch.bool, device="cuda")
        mask[..., int(0.9 * Lkv):] = False
    elif a.mask == "additive":
        gen = torch.Generator(device="cpu").manual_seed(6)
        mask = torch.randn(a.L, Lkv, generator=gen).to(q.dtype).cuda()
    path = {"auto": _lib.PATH_AUTO, "tensor": _lib.PATH_TENSOR, "simt": _lib.PATH_SIMT,
            "vector": _lib.PATH_VECTOR}[a.path]
    with api.force_path(path):
        out, lse = api.attention_forward(q, k, v, scale=scale, is_causal=a.causal, attn_mask=mask)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ws = torch.empty(max(16, api.workspace_bytes(q, k)), device="cuda", dtype=torch.uint8)

        def once():
            if a.op in ("fwd", "step"):
                api.attention_forward(q, k, v, scale=scale, is_causal=a.causal, out=out, lse=lse,
                                      attn_mask=mask)
            if a.op in ("bwd", "step"):
                api.attention_backward(q, k, v, out, do, lse, scale=scale, is_causal=a.causal,
                                       workspace=ws, dq=dq, dk=dk, dv=dv, attn_mask=mask)

        ms = timed(once, a.iters)
    f = 4.0 * a.B * a.Hq * a.L * (a.Lkv or a.L) * a.D * (0.5 if a.causal else 1.0)
    mult = {"fwd": 1.0, "bwd": 2.5, "step": 3.5}[a.op]
    print(f"{a.op}: {ms:.4f} ms per call, {mult * f / ms / 1e9:.1f} TFLOP/s")


if __name__ == "__main__":
    main()
