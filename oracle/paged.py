"""Plain fp64 oracle of the 16-bit paged cache: TEST INFRASTRUCTURE ONLY, like the rest of the
package.  Sequences are given as lists of keys and values [Hkv, n_b, D], row by row."""
from __future__ import annotations

import numpy as np


def limits(n, L, count, causal):
    """How many tokens each of L rows of a sequence of n sees; the last `count` rows are real."""
    pos = n - L + np.arange(L)
    seen = np.maximum(pos + 1, 0) if causal else np.full(L, n)
    return np.where(np.arange(L) >= L - min(max(count, 0), L), seen, 0)


def attention(q, ks, vs, scale, causal, counts=None, sinks=None):
    """(O, lse, A, S) of q [B,Hq,L,D]; A = sum_j w_j·|v_j| and S [B,Hq,L] = the largest
    sum_d |q_d·k_jd|·|scale| of a row: what rounding errors of the output and the scores grow with."""
    B, Hq, L, D = q.shape
    O, A = np.zeros(q.shape), np.zeros(q.shape)
    lse, S = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    for b in range(B):
        H, n = ks[b].shape[:2]
        lim = limits(n, L, L if counts is None else counts[b], causal)
        for h in range(Hq):
            g = h // (Hq // H)
            sink = -np.inf if sinks is None else float(sinks[h])
            for i in range(L):
                e = lim[i]
                s = scale * (ks[b][g, :e] @ q[b, h, i])
                top = max(s.max(initial=-np.inf), sink)
                if top == -np.inf:
                    continue
                p = np.exp(s - top)
                total = p.sum() + np.exp(sink - top)
                O[b, h, i] = p @ vs[b][g, :e] / total
                A[b, h, i] = p @ np.abs(vs[b][g, :e]) / total
                lse[b, h, i] = top + np.log(total)
                S[b, h, i] = abs(scale) * (np.abs(ks[b][g, :e]) @ np.abs(q[b, h, i])).max(initial=0)
    return O, lse, A, S


def weights(q, ks, lse, old, scale, causal, counts=None):
    """(weights [B,Hkv,slots] after the call, the gain alone)."""
    B, Hq, L, _ = q.shape
    out, gain = old.copy(), np.zeros(old.shape)
    for b in range(B):
        H, n = ks[b].shape[:2]
        count = L if counts is None else min(max(counts[b], 0), L)
        lim = limits(n, L, count, causal)
        out[b, :, max(n - count, 0):n] = 0
        for h in range(Hq):
            g = h // (Hq // H)
            for i in range(L):
                if lse[b, h, i] != -np.inf:
                    gain[b, g, :lim[i]] += np.exp(scale * (ks[b][g, :lim[i]] @ q[b, h, i]) - lse[b, h, i])
    return out + gain, gain


def kept(weights, n, budget, recent):
    """Positions that stay of one row of weights of n tokens, by sorting (position, weight) pairs."""
    if n <= budget:
        return list(range(n))
    old = n - recent

    def order(j):
        w = weights[j]
        return (1, 0.0, j) if np.isnan(w) else (0, -w, j)

    return sorted(sorted(range(old), key=order)[:budget - recent]) + list(range(old, n))
