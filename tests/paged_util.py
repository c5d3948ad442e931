"""Shared by the tests of the 16-bit paged cache."""
import numpy as np
import torch

from cache_util import TYPES, draw_rows, ints, make_table
from oracle import paged as ref
from scaled_dot_product_flash_gb300 import api
from scaled_dot_product_flash_gb300.inputs import as_f64

NAN = float("nan")


def dirty(pages, H, page, D, dtype):
    """A cache of nothing but NaN."""
    return api.paged_empty(pages, H, page, D, TYPES[dtype]).fill_(NAN)


def fill(rng, lens, H, D, page, dtype, width=None, spread=1.0):
    """A cache holding random keys and values of these lengths (NaN elsewhere), its table, and
    each sequence's fp64 keys and values; put there by torch, page by page."""
    table, pages = make_table(rng, lens, page, width)
    cache = torch.full((pages, 2, H, page, D), NAN, dtype=TYPES[dtype])
    rows = []
    for b, n in enumerate(lens):
        kv = draw_rows(rng, (2, H, n, D), dtype, spread)
        kv[0] += torch.from_numpy(rng.standard_normal((H, 1, D))).to(kv.dtype)   # channels off zero
        for j in range(0, n, page):
            m = min(page, n - j)
            cache[table[b, j // page], :, :, :m] = kv[:, :, j:j + m]
        rows.append(as_f64(kv))
    return cache.cuda(), table, [x[0] for x in rows], [x[1] for x in rows]


def check(out, lse, q, ks, vs, scale, causal, dtype, counts=None, sinks=None, few=None):
    """Tolerances, T the element type, u = 2^-24:
    o: eps(T)/2·|o|        its rounding (half a step of the smallest numbers in fp16)
     + eps(T)/2·A          P rounded to T before it meets V (A = sum_j w_j·|v_j|); 2·(eps(T)/2)^2·A
                           where the remainder follows it, as it does for few rows (`few`)
     + 2·ds·A + n·2u·A     the scores' errors move each weight and the sum by ds = (D + 8)·u·S
                           relative to themselves, S the row's largest sum of |q·k|·scale, and the
                           exponential by another 2^-21; sums of n terms in fp32, which an MMA may
                           cut off instead of rounding
    lse: ds + n·u + 2^-21 + 2^-22·|lse|"""
    o, want, A, S = ref.attention(as_f64(q), ks, vs, scale, causal, counts, sinks)
    D, u = q.shape[3], 2.0**-24
    n = max([1] + [k.shape[1] for k in ks])
    few = q.shape[1] // ks[0].shape[0] * q.shape[2] <= 32 if few is None else few
    half = torch.finfo(TYPES[dtype]).eps / 2
    ds = (D + 8) * u * S + 2.0**-21
    tol = half * np.abs(o) + (2 * half**2 if few else half) * A + (2 * ds[..., None] + 2 * n * u) * A + (2.0**-25 if dtype == "f16" else 1e-38)
    got = as_f64(out)
    assert np.isfinite(got).all()
    worst = (np.abs(got - o) / tol).max()
    assert worst <= 1, f"out is {worst:.2f} of its tolerance"
    if lse is not None:
        got, none = as_f64(lse), np.isneginf(want)
        assert np.array_equal(np.isneginf(got), none)
        off = np.abs(np.where(none, 0, got) - np.where(none, 0, want)) / (ds + n * u + 2.0**-21 + 2.0**-22 * np.abs(np.where(none, 0, want)))
        assert off.max() <= 1, f"lse is {off.max():.2f} of its tolerance"


def on_device(table, lens, counts=None):
    return (table.cuda(), ints(lens).cuda()), None if counts is None else ints(counts).cuda()
