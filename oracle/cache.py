"""Plain fp64 oracle of the rotary embedding and of the 4-bit paged cache: TEST
INFRASTRUCTURE ONLY, like the rest of the package.

Rotary: pair p of a row is the complex number x_a + i·x_b; it is multiplied by
exp(i·position·inv_freq[p]).

Cache: groups of 32 elements of a row with z = min and s = (max − z)/15, both rounded to the
element type (the quotient is taken in fp32, as the format says), and codes round((x − z)/s)
to even, 0 where s is 0.  A group with an element that is not finite, or whose range
overflows fp32, has s = 0, z = NaN and codes 0.  Tiles are packed element by element from
the documented word formulas.
"""
from __future__ import annotations

import numpy as np
import torch

from .ref import sdpa_forward

GROUP, TILE = 32, 16


def rotary(x, positions, inv_freq, axes=None, adjacent=False, inverse=False):
    """x [B,H,L,D] fp64; positions [A,B,L] integers; inv_freq [R/2]; axes [R/2] or None."""
    x = np.array(x, dtype=np.float64)
    n = len(inv_freq)
    axes = np.zeros(n, dtype=int) if axes is None else np.asarray(axes)
    for p in range(n):
        angle = positions[axes[p]].astype(np.float64) * float(inv_freq[p])
        w = np.exp(1j * (-angle if inverse else angle))[:, None, :]
        a, b = (2 * p, 2 * p + 1) if adjacent else (p, p + n)
        z = (x[..., a] + 1j * x[..., b]) * w
        x[..., a], x[..., b] = z.real, z.imag
    return x


def rounded(x, dtype):
    """fp64 values rounded to a torch dtype, as fp64."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).double().numpy()


def quantise(x, dtype):
    """(codes [..., D], s [..., D/32], z [..., D/32]) of rows x [..., D] (fp64 holding dtype)."""
    g = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    with np.errstate(invalid="ignore", over="ignore"):
        z, high = g.min(-1), g.max(-1)
        spread = (high.astype(np.float32) - z.astype(np.float32)).astype(np.float32)
        bad = ~np.isfinite(g).all(-1) | ~np.isfinite(spread)
        s = rounded((spread / np.float32(15)).astype(np.float64), dtype)
        s, z = np.where(bad, 0.0, s), np.where(bad, np.nan, z)
        q = np.where((s > 0)[..., None], (g - z[..., None]) / np.where(s > 0, s, 1.0)[..., None], 0.0)
    code = np.minimum(np.rint(q), 15).astype(np.uint8)
    return code.reshape(x.shape), s, z


def values(code, s, z):
    g = code.reshape(*code.shape[:-1], code.shape[-1] // GROUP, GROUP).astype(np.float64)
    return (z[..., None] + s[..., None] * g).reshape(code.shape)


def word_places(D):
    """For every (row, element) of a tile: byte and shift of its K code and its V code, and for
    every (row, group) the byte of its (s, z) pair counted from the parameters' start."""
    W = min(D // GROUP, 4)
    JB = D // GROUP // W
    k, v, p = {}, {}, {}
    for r in range(TILE):
        for d in range(D):
            j, e = divmod(d, GROUP)
            t, n = divmod(e, 8)
            word = (((r // 8 * JB + j // W) * 8 + r % 8) * 4 + t) * W + j % W
            k[r, d] = (4 * word + n // 2, 4 * (n % 2))
            g, n = divmod(e, 4)
            word = (((r // 8 * JB + j // W) * 8 + g) * 4 + r % 8 // 2) * W + j % W
            v[r, d] = (8 * D + 4 * word + 2 * (r % 2) + n // 2, 4 * (n % 2))
        for j in range(D // GROUP):
            p[r, j] = 4 * ((j // W * TILE + r) * W + j % W)
    return k, v, p


def put_token(tile, r, places, k, v, dtype):
    """Writes one token's rows k and v [D] into place r of a tile (uint8 [20·D], in place)."""
    D = tile.shape[0] // 20
    for x, where, at in ((k, places[0], 16 * D), (v, places[1], 18 * D)):
        code, s, z = quantise(x, dtype)
        for d in range(D):
            byte, shift = where[r, d]
            tile[byte] = (int(tile[byte]) & ~(15 << shift)) | (int(code[d]) << shift)
        bits = torch.from_numpy(np.stack([s, z], -1)).to(dtype).view(torch.uint8).numpy().reshape(-1, 4)
        for j in range(D // GROUP):
            o = at + places[2][r, j]
            tile[o:o + 4] = bits[j]


def cached_attention(q, ks, vs, scale, causal, sinks=None):
    """(O, lse) of q [B,Hq,L,D] over per-sequence keys and values [Hkv, n_b, D] (n_b may be 0);
    causal: query i sees positions up to n_b − L + i."""
    O, lse = np.zeros_like(q), np.full(q.shape[:3], -np.inf)
    B, Hq, L, _ = q.shape
    for b in range(B):
        n = ks[b].shape[1]
        for i in range(L):
            end = n - L + i + 1 if causal else n
            if end <= 0:
                if sinks is not None:
                    lse[b, :, i] = sinks
                continue
            O[b:b + 1, :, i:i + 1], lse[b:b + 1, :, i:i + 1] = sdpa_forward(
                q[b:b + 1, :, i:i + 1], ks[b][None, :, :end], vs[b][None, :, :end], scale, False,
                sinks=sinks)
    return O, lse
