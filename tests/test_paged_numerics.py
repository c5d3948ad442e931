"""What attention over a 16-bit paged cache makes of weights, scores and values at the ends of their
ranges, against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

from cache_util import TYPES, draw_rows, ints, make_table
from oracle import paged as ref
from paged_util import NAN, check, fill, on_device
from scaled_dot_product_flash_gb300 import _lib, api
from scaled_dot_product_flash_gb300.inputs import as_f64
from test_paged_evict import check_weights


def put(ks, vs, page, dtype, rng):
    """(cache, table) holding these keys and values [Hkv, n, D], NaN elsewhere."""
    lens = [k.shape[1] for k in ks]
    table, pages = make_table(rng, lens, page)
    H, _, D = ks[0].shape
    cache = torch.full((pages, 2, H, page, D), NAN, dtype=TYPES[dtype])
    for b, n in enumerate(lens):
        for j in range(0, n, page):
            m = min(page, n - j)
            cache[table[b, j // page], 0, :, :m] = ks[b][:, j:j + m]
            cache[table[b, j // page], 1, :, :m] = vs[b][:, j:j + m]
    return cache.cuda(), table


# ---- weights far below a row's largest

FORMS = [(64, 1, 1), (128, 4, 8), (64, 1, 60), (128, 2, 200), (256, 1, 1), (256, 1, 20), (256, 1, 50)]  # D, G, L: every kernel


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("gap", [6, 12, 17.5, 20, 30, 60])
@pytest.mark.parametrize("n,heavy", [(90, [0]), (4096, [0]), (2500, [3, 700, 1500, 2300])])
@pytest.mark.parametrize("D,G,L", FORMS)
def test_small_weights_are_kept(D, G, L, n, heavy, gap, dtype):
    """A few tokens that score `gap` above all others and have a value of 0, as attention sinks do: what
    comes out is what the others contribute.  Tolerances as in paged_util.check, and for what P in T keeps of
    a weight (paged.h):
      2^-25·max|v|   fp16: tokens in a heavy one's tile of at most 128 are off by 2^-32 of it each, and
                     the heavy ones' weights together are 1 at most
      2^-16·A        fp16: all others by 2^-18 of their tile's largest, which is at most e^1 = 2^1.45
                     times a weight here"""
    if n < L:
        pytest.skip("rows past the first token")
    rng = np.random.default_rng(int(10 * gap) + n + D)
    k = torch.zeros(1, n, D, dtype=TYPES[dtype])
    k[0, :, 0] = torch.from_numpy(rng.uniform(-0.4, 0.4, n)).to(k.dtype)
    k[0, :, 1:] = draw_rows(rng, (n, D - 1), dtype)
    v = draw_rows(rng, (1, n, D), dtype, 0.25) + 1
    k[0, heavy, 0] = gap
    v[0, heavy] = 0
    cache, table = put([k], [v], 32, dtype, rng)
    q = torch.zeros(1, G, L, D, dtype=TYPES[dtype])
    q[..., 0] = 1                                                                # a score is a key's first element
    at, _ = on_device(table, [n])
    out, lse = api.paged_attention(q.cuda(), cache, *at, scale=1.0, need_lse=True)
    api.poll_status()
    o, want, A, S = ref.attention(as_f64(q), [as_f64(k)], [as_f64(v)], 1.0, True)
    half, u = torch.finfo(TYPES[dtype]).eps / 2, 2.0**-24
    ds = (D + 8) * u * S[..., None] + 2.0**-21
    p = (2 * half**2 if G * L <= 32 else half) + (2.0**-16 if dtype == "f16" else 0)
    floor = 2.0**-25 * (1 + as_f64(v).max()) if dtype == "f16" else 1e-38
    tol = half * np.abs(o) + (p + 2 * ds + 2 * n * u) * A + floor
    worst = (np.abs(as_f64(out) - o) / tol).max()
    assert worst <= 1, f"out is {worst:.2f} of its tolerance"
    off = np.abs(as_f64(lse) - want) / (ds[..., 0] + n * u + 2.0**-21 + 2.0**-22 * np.abs(want))
    assert off.max() <= 1, f"lse is {off.max():.2f} of its tolerance"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("slope", [0.02, -0.02])
@pytest.mark.parametrize("D,G,L", FORMS)
def test_scores_that_rise_and_fall(D, G, L, slope, dtype):
    """4000 scores on a line from 0 to 80, up or down: bases move every few tiles.  Tolerances as in
    test_small_weights_are_kept; in fp16 2^-25·max|v| is for the tokens before a base moves on, 500 of them
    at most (10 on a scale where the row's largest weight is 1), off by 2^-32 of the row's largest, which is a
    fiftieth of its sum (1 / (1 - e^-0.02))."""
    rng = np.random.default_rng(5)
    n = 4000
    k = torch.zeros(1, n, D, dtype=TYPES[dtype])
    line = slope * np.arange(n)
    k[0, :, 0] = torch.from_numpy(np.round(line)).to(k.dtype)                    # whole numbers to 80 are exact
    k[0, :, 1] = torch.from_numpy(line - np.round(line)).to(k.dtype)
    v = draw_rows(rng, (1, n, D), dtype)
    cache, table = put([k], [v], 64, dtype, rng)
    q = torch.zeros(1, G, L, D, dtype=TYPES[dtype])
    q[..., :2] = 1
    at, _ = on_device(table, [n])
    out, lse = api.paged_attention(q.cuda(), cache, *at, scale=1.0, need_lse=True)
    api.poll_status()
    o, want, A, S = ref.attention(as_f64(q), [as_f64(k)], [as_f64(v)], 1.0, True)
    half, u = torch.finfo(TYPES[dtype]).eps / 2, 2.0**-24
    ds = (D + 8) * u * S[..., None] + 2.0**-21
    p = 2 * half**2 if G * L <= 32 else half
    tol = half * np.abs(o) + (p + 2 * ds + 2 * n * u) * A + 2.0**-25 * (1 + np.abs(as_f64(v)).max())
    worst = (np.abs(as_f64(out) - o) / tol).max()
    assert worst <= 1, f"out is {worst:.2f} of its tolerance"
    assert (np.abs(as_f64(lse) - want) / (ds[..., 0] + n * u + 2.0**-21 + 2.0**-22 * np.abs(want))).max() <= 1


# ---- scores up to 2^26


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("steps", [[0], [-32, 0], [0, -64, 0]])
@pytest.mark.parametrize("D,G,L", FORMS)
def test_large_scores(D, G, L, steps, dtype):
    """Scores of 5.7e7, where fp32 counts in steps of 4 and of 8 once log2(e) is in: equal ones have equal
    weights, whole steps less none.  Tolerance: the output's rounding, P's, the exponential's 2^-21 and the
    sums' n·2^-23."""
    rng = np.random.default_rng(8)
    n = 1500
    k = torch.zeros(1, n, D, dtype=TYPES[dtype])
    for x, step in enumerate(steps):                                             # one part of the tokens each
        k[0, n * x // len(steps):, 0] = 60224 + 32 * step
    v = draw_rows(rng, (1, n, D), dtype, 0.2) + 1
    cache, table = put([k], [v], 48, dtype, rng)
    q = torch.zeros(1, G, L, D, dtype=TYPES[dtype])
    q[..., 0] = 948
    at, _ = on_device(table, [n])
    out, lse = api.paged_attention(q.cuda(), cache, *at, scale=1.0, need_lse=True)
    api.poll_status()
    o, want, A, _ = ref.attention(as_f64(q), [as_f64(k)], [as_f64(v)], 1.0, True)
    half = torch.finfo(TYPES[dtype]).eps / 2
    tol = half * np.abs(o) + ((2 * half**2 if G * L <= 32 else half) + 2.0**-21 + 2 * n * 2.0**-24) * A
    worst = (np.abs(as_f64(out) - o) / tol).max()
    assert worst <= 1, f"out is {worst:.2f} of its tolerance"
    assert (np.abs(as_f64(lse) - want) <= 2.0**-22 * np.abs(want)).all()


# ---- values that are not finite


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("what", [NAN, float("inf")])
@pytest.mark.parametrize("D,G,L", [f for f in FORMS if f[2] > 1] + [(64, 1, 2), (128, 1, 5), (256, 2, 4)])
def test_a_hidden_value_where_every_score_is_minus_infinity(D, G, L, what, dtype):
    """Rows that see nothing but scores of -inf rest at 0 and -inf, whatever a token that they do not see holds."""
    rng = np.random.default_rng(9)
    n = L + 5
    k = torch.zeros(1, n, D, dtype=TYPES[dtype])
    k[0, :-1, 0] = -math.inf
    v = draw_rows(rng, (1, n, D), dtype)
    v[0, -1] = what
    cache, table = put([k], [v], 32, dtype, rng)
    q = torch.zeros(1, G, L, D, dtype=TYPES[dtype])
    q[..., 0] = 1
    at, _ = on_device(table, [n])
    out, lse = api.paged_attention(q.cuda(), cache, *at, scale=1.0, need_lse=True)
    api.poll_status()
    assert not out[:, :, :-1].any() and torch.isneginf(lse[:, :, :-1]).all()
    assert not out[:, :, -1].isfinite().any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,G,L", FORMS)
def test_some_values_that_are_not_finite(D, G, L, dtype):
    """NaN and infinities strewn over the values, many in columns of their own, some with others: what a row
    sees decides, column by column, over several chunks and pages.  Tolerance of the rest: paged_util.check's
    terms, P to 2^-20 where a column was mended."""
    rng = np.random.default_rng(10)
    n = 3000
    k = draw_rows(rng, (1, n, D), dtype, 0.5)
    v = draw_rows(rng, (1, n, D), dtype)
    bad = torch.zeros(n, D)
    for j in [0, 17, 300, 1500, *range(n - 40, n, 3)]:
        for x in rng.choice(D, 3, replace=False):
            bad[j, x] = [NAN, math.inf, -math.inf][rng.integers(3)]
    v[0] = torch.where(bad != 0, bad.to(v.dtype), v[0])
    cache, table = put([k], [v], 48, dtype, rng)
    q = draw_rows(rng, (1, G, L, D), dtype, 0.5)
    at, _ = on_device(table, [n])
    out, lse = api.paged_attention(q.cuda(), cache, *at, need_lse=True)
    api.poll_status()
    clean = torch.where(bad != 0, 0, v[0].double())[None].numpy()
    o, want, A, S = ref.attention(as_f64(q), [as_f64(k)], [clean], D**-0.5, True)
    marks = bad.double().numpy()
    for i in range(L):
        seen = marks[:n - L + i + 1]
        nan, up, down = np.isnan(seen).any(0), (seen == np.inf).any(0), (seen == -np.inf).any(0)
        o[:, :, i] = np.where(nan | (up & down), np.nan, np.where(up, np.inf, np.where(down, -np.inf, o[:, :, i])))
    got = as_f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(o)) and np.array_equal(got[np.isinf(o)], o[np.isinf(o)])
    half, u = torch.finfo(TYPES[dtype]).eps / 2, 2.0**-24
    tol = half * np.abs(o) + (max(2.0**-20, 2 * half**2 if G * L <= 32 else half) + 2 * (D + 8) * u * S[..., None] + 2.0**-20 + 2 * n * u) * A + 2.0**-25
    fine = np.isfinite(o)
    assert (np.abs(got - o)[fine] <= tol[fine]).all() and torch.isfinite(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("what", [NAN, math.inf])
@pytest.mark.parametrize("G,L,D", [(4, 60, 64), (4, 300, 128), (2, 40, 256), (4, 8, 64), (4, 2, 128)])
def test_a_hidden_value_costs_little(G, L, D, what):
    """One token of 16000 with values that are not finite, which all rows but the last do not see: no more
    than 600 times a call's time."""
    rng = np.random.default_rng(35)
    n = 16000
    cache, table, _, _ = fill(rng, [n], 2, D, 64, "bf16")
    q = draw_rows(rng, (1, 2 * G, L, D), "bf16").cuda()
    at, _ = on_device(table, [n])

    def timed():
        api.paged_attention(q, cache, *at)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        out, _ = api.paged_attention(q, cache, *at)
        b.record()
        b.synchronize()
        return out, a.elapsed_time(b)

    good, plain = timed()
    cache[table[0, (n - 1) // 64], 1, :, (n - 1) % 64] = what
    out, slow = timed()
    api.poll_status()
    assert not out[:, :, -1].isfinite().any()
    assert (out[:, :, :-1].float() - good[:, :, :-1].float()).abs().max() <= 2.0**-8 * good.float().abs().max() + 2.0**-8
    assert slow < 600 * max(plain, 0.05)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,size", [("bf16", 2.0**100), ("f16", 60000.0)])
@pytest.mark.parametrize("D,G,L", FORMS)
def test_large_values(D, G, L, dtype, size):
    """Values whose sum over 4000 tokens is far from fp32's end in bf16, and near fp16's largest number.
    Tolerance: paged_util.check's terms; A is at most `size`."""
    rng = np.random.default_rng(11)
    n = 4000
    k = draw_rows(rng, (1, n, D), dtype, 0.5)
    v = torch.from_numpy(size * rng.choice([1, -0.5], (1, n, D))).to(k.dtype)
    v[..., 0] = size
    cache, table = put([k], [v], 48, dtype, rng)
    q = draw_rows(rng, (1, G, L, D), dtype, 0.5)
    at, _ = on_device(table, [n])
    out, _ = api.paged_attention(q.cuda(), cache, *at)
    api.poll_status()
    o, _, A, S = ref.attention(as_f64(q), [as_f64(k)], [as_f64(v)], D**-0.5, True)
    half, u = torch.finfo(TYPES[dtype]).eps / 2, 2.0**-24
    tol = half * np.abs(o) + ((2 * half**2 if G * L <= 32 else half) + 2 * (D + 8) * u * S[..., None] + 2.0**-20 + 2 * n * u) * A
    assert (np.abs(as_f64(out) - o) <= tol).all()


# ---- forms and arguments that other tests do not reach


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,Hq,Hkv,L,page,lens,counts", [
    ("bf16", 4, 1, 5, 16, [300, 9, 5], [5, 2, 0]),
    ("f16", 17, 1, 1, 48, [700, 1], None),
    ("bf16", 8, 2, 8, 64, [129, 500], [8, 3]),
    ("f16", 2, 1, 16, 32, [1300, 16, 40], [16, 16, 7]),
])
def test_17_to_32_rows_at_head_dim_256(dtype, Hq, Hkv, L, page, lens, counts, causal):
    """One tile of rows, head and remainder of P in every tile; weights in two passes over the rows."""
    rng = np.random.default_rng(12 + L)
    cache, table, ks, vs = fill(rng, lens, Hkv, 256, page, dtype)
    q = draw_rows(rng, (len(lens), Hq, L, 256), dtype, 1.5)
    at, dev_counts = on_device(table, lens, counts)
    how = dict(is_causal="bottom_right" if causal else False, counts=dev_counts)
    out, lse = api.paged_attention(q.cuda(), cache, *at, need_lse=True, **how)
    check(out, lse, q, ks, vs, 1 / 16, causal, dtype, counts)
    old = torch.from_numpy(rng.random((len(lens), Hkv, max(lens) + 5))).float()
    got = api.paged_weights(q.cuda(), cache, *at, lse, old.cuda(), **how)
    api.poll_status()
    check_weights(got, q, ks, vs, lse, old, 1 / 16, causal, counts)


@pytest.mark.gpu
@pytest.mark.parametrize("L,counts", [(70, [70, 33]), (33, None)])
def test_weights_under_a_table_of_8_million_tokens(L, counts):
    """More blocks of keys than a grid's second dimension: the kernel for few rows, in several passes over them."""
    rng = np.random.default_rng(13)
    lens = [300, 71]
    cache, table, ks, vs = fill(rng, lens, 1, 32, 65536, "bf16", width=129)
    q = draw_rows(rng, (2, 2, L, 32), "bf16")
    at, dev_counts = on_device(table, lens, counts)
    out, lse = api.paged_attention(q.cuda(), cache, *at, need_lse=True, counts=dev_counts, max_len=300)
    old = torch.rand(2, 1, 8454144, generator=torch.Generator().manual_seed(1))
    got = api.paged_weights(q.cuda(), cache, *at, lse, old.cuda(), counts=dev_counts)
    api.poll_status()
    assert torch.equal(got[:, :, 300:].cpu(), old[:, :, 300:])
    check_weights(got[:, :, :320], q, ks, vs, lse, old[:, :, :320], 32**-0.5, True, counts)


@pytest.mark.gpu
@pytest.mark.parametrize("L", [1, 60, 200])
def test_strides_of_single_dimensions_do_not_matter(L):
    """The largest batch stride that is valid, of a batch of one."""
    rng = np.random.default_rng(14)
    cache, table, ks, vs = fill(rng, [250], 1, 64, 16, "bf16")
    q = draw_rows(rng, (1, 1, L, 64), "bf16").cuda()
    out = torch.empty_like(q)
    lse = torch.empty(1, 1, L, device="cuda")
    at, _ = on_device(table, [250])
    c, far = api._paged(cache, *at, 1), 1 << 40
    need = _lib.sdpa_paged_attn_workspace_size(c, 1, 1, L, 0)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    lay = _lib.Int64x6(far, far, 64, far, far, 64)
    assert _lib.sdpa_paged_attn(c, q.data_ptr(), out.data_ptr(), lse.data_ptr(), None, lay, None, 1, 1, L, 0.125, 2, 0, ws.data_ptr(), need, stream) == 0
    w = torch.zeros(1, 1, 250, device="cuda")
    strides = api._pack2(far, far)
    assert _lib.sdpa_paged_weights(c, q.data_ptr(), lse.data_ptr(), w.data_ptr(), strides, 250, _lib.Int64x3(far, far, 64), None, 1, 1, L, 0.125, 2, 0, stream) == 0
    api.poll_status()
    check(out, lse, q, ks, vs, 0.125, True, "bf16")
    assert abs(w.sum().item() - L) < 1e-3
