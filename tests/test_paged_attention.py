"""Writing a 16-bit paged cache and attention over it, against the fp64 oracle (tolerances:
paged_util.check)."""
import math

import numpy as np
import pytest
import torch

from cache_util import TYPES, draw_rows, ints, make_table
from oracle import paged as ref
from paged_util import NAN, check, dirty, fill, on_device
from scaled_dot_product_flash_gb300 import _lib, api, build
from scaled_dot_product_flash_gb300.inputs import as_f64

INVALID, UNSUPPORTED, WORKSPACE, INDEX = 1, 2, 5, 6

# ---- without a GPU: fake, 16-byte aligned addresses; every case is refused before a launch

DATA, TABLE, LENS, Q, OUT, LSE, SINKS, WS, COUNTS = (0x10000000 * (n + 1) for n in range(9))
GOOD = dict(data=DATA, num_pages=4, page_size=32, Hkv=2, D=64, dtype=2, pages=TABLE, pages_stride=300, pages_per_seq=300, lens=LENS)
BAD_CACHES = [
    (dict(data=0), INVALID), (dict(data=DATA + 8), INVALID), (dict(pages=0), INVALID), (dict(lens=0), INVALID), (dict(pages=TABLE + 2), INVALID),
    (dict(lens=LENS + 1), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=24), INVALID), (dict(page_size=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(pages_stride=1), INVALID), (dict(pages_per_seq=0), INVALID), (dict(D=48), UNSUPPORTED), (dict(dtype=0), UNSUPPORTED),
    (dict(page_size=131072), UNSUPPORTED), (dict(page_size=65536, pages_per_seq=32768, pages_stride=32768), UNSUPPORTED),
    (dict(page_size=65536, Hkv=32768, D=256), UNSUPPORTED), (dict(B=0), INVALID), (dict(B=70000), UNSUPPORTED)]


def cache_of(a):
    build.build()
    return _lib.Cache(*(a[n] for n in GOOD))


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(L=0), INVALID), (dict(B=60000, L=60000), UNSUPPORTED), (dict(k=0), INVALID), (dict(v=OUT + 2), INVALID), (dict(lay=None), INVALID),
    (dict(lay=(4096, 2048, 64, 4096, 0, 64)), INVALID), (dict(lay=(4096, 2048, 68, 4096, 2048, 64)), INVALID), (dict(k=DATA + 64), INVALID),
    (dict(counts=COUNTS + 2), INVALID), (dict(counts=DATA + 4), INVALID), (dict(lens=DATA), INVALID), (dict(pages=DATA + 16), INVALID)])
def test_write_refused(kw, code):
    a = dict(GOOD, B=2, L=5, k=Q, v=OUT, counts=None, lay=(4096, 2048, 64, 4096, 2048, 64))
    a.update(kw)
    lay = None if a["lay"] is None else _lib.Int64x6(*a["lay"])
    assert _lib.sdpa_paged_write(cache_of(a), a["k"], a["v"], lay, a["counts"], a["B"], a["L"], None) == code


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(q=0), INVALID), (dict(out=0), INVALID), (dict(q=Q + 8), INVALID), (dict(lse=LSE + 4), INVALID), (dict(sinks=SINKS + 2), INVALID),
    (dict(counts=COUNTS + 1), INVALID), (dict(lay=None), INVALID), (dict(lay=(256, 64, 60, 256, 64, 64)), INVALID),
    (dict(lay=(0, 64, 64, 256, 64, 64)), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=NAN), INVALID), (dict(causal=3), INVALID),
    (dict(causal=-1), INVALID), (dict(causal=1), UNSUPPORTED), (dict(Hq=3), INVALID), (dict(Hq=0), INVALID), (dict(Lq=0), INVALID),
    (dict(Hq=70000), UNSUPPORTED), (dict(out=Q), INVALID), (dict(lse=OUT), INVALID), (dict(out=DATA), INVALID), (dict(out=SINKS - 16), INVALID),
    (dict(lse=TABLE), INVALID), (dict(out=LENS), INVALID), (dict(out=COUNTS), INVALID)])
def test_attention_refused(kw, code):
    a = dict(GOOD, q=Q, out=OUT, lse=LSE, sinks=SINKS, counts=COUNTS, lay=(256, 64, 64, 256, 64, 64), B=2, Hq=4, Lq=1, scale=0.125, causal=2)
    a.update(kw)
    lay = None if a["lay"] is None else _lib.Int64x6(*a["lay"])
    assert _lib.sdpa_paged_attn(cache_of(a), a["q"], a["out"], a["lse"], a["sinks"], lay, a["counts"], a["B"], a["Hq"], a["Lq"], a["scale"], a["causal"], 0,
                                WS, 1 << 26, None) == code


def test_sizes():
    build.build()
    assert _lib.sdpa_paged_page_bytes(64, 8, 128, 2) == 2 * 8 * 64 * 128 * 2
    assert _lib.sdpa_paged_page_bytes(24, 8, 128, 2) == 0 and _lib.sdpa_paged_page_bytes(64, 8, 128, 0) == 0
    with pytest.raises(ValueError):
        api.paged_empty(2, 1, 8, 64, device="cpu")
    cache = api.paged_empty(3, 2, 16, 64, torch.float16, device="cpu")
    assert tuple(cache.shape) == (3, 2, 2, 16, 64)
    k = torch.zeros(1, 2, 3, 64, dtype=torch.float16)
    with pytest.raises(ValueError):                                              # host tensors
        api.paged_write(cache, k, k, ints([[0]]), ints([3]))
    with pytest.raises(ValueError):
        api.paged_attention(k, cache, ints([[0]]), ints([3]))


@pytest.mark.parametrize("B,Hq,Hkv,L,D", [(1, 32, 8, 4096, 128), (1, 32, 8, 512, 128), (1, 4, 1, 1, 128), (4096, 32, 8, 1, 64), (64, 64, 1, 1, 256), (1, 9, 3, 100, 96)])
@pytest.mark.parametrize("tokens", [2048, 131072, 1 << 30])
def test_the_workspace_stays_small(B, Hq, Hkv, L, D, tokens):
    build.build()
    c = _lib.Cache(DATA, 4, 1 << 15, Hkv, D, 2, TABLE, 1 << 15, max(1, tokens >> 15), LENS)
    assert _lib.sdpa_paged_attn_workspace_size(c, B, Hq, L, tokens) <= max(64 << 20, B * Hq * L * (D + 2) * 4)


def test_oracle_agrees_with_the_dense_one():
    from oracle import ref as dense

    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 2, 9, 8))
    q = rng.standard_normal((1, 4, 9, 8))
    o, lse, A, _ = ref.attention(q, [k], [v], 0.3, True)
    want = dense.sdpa_forward(q, k[None], v[None], 0.3, True)
    assert np.allclose(o, want[0]) and np.allclose(lse, want[1]) and (A >= np.abs(o) - 1e-12).all()
    # a call of 9 rows of which 4 are real is a call of those 4
    part = ref.attention(q, [k], [v], 0.3, True, counts=[4])
    assert not part[0][:, :, :5].any() and np.allclose(part[0][:, :, 5:], o[:, :, 5:]) and np.isneginf(part[1][:, :, :5]).all()
    # the weights of a step sum to the number of rows
    w, gain = ref.weights(q, [k], lse, np.full((1, 2, 12), 7.0), 0.3, True)
    assert np.allclose(gain.sum(), 4 * 9) and (w[..., 9:] == 7).all() and np.allclose(w[..., :9], gain[..., :9])
    assert ref.kept(np.array([3, 1, 3, NAN, 0.0, -0.0, 2, 9]), 8, 5, 1) == [0, 1, 2, 6, 7]
    assert ref.kept(np.array([1, 1, 1, 1.0]), 4, 2, 0) == [0, 1] and ref.kept(np.array([1, 1.0]), 2, 2, 1) == [0, 1]


# ---- on the GPU


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,H,L,D,page,lens,counts", [
    ("bf16", 1, 1, 32, 16, [1], None),
    ("bf16", 2, 1, 128, 16, [1, 16, 17, 100], None),
    ("f16", 3, 21, 96, 48, [21, 50, 5, 0], [21, 2, 21, 21]),       # padding, a short sequence, an empty one
    ("f16", 1, 40, 64, 32, [40, 47, 64], [0, 40, 17]),
    ("bf16", 2, 7, 256, 16, [7, 9, 33], [-3, 9, 1]),               # counts outside 0..L
    ("bf16", 2, 335, 128, 64, [400, 336], None),
])
@pytest.mark.parametrize("tokens_first", [False, True])
def test_write(dtype, H, L, D, page, lens, counts, tokens_first):
    rng = np.random.default_rng(L + D)
    table, pages = make_table(rng, lens, page)
    cache = dirty(pages, H, page, D, dtype)
    k, v = (draw_rows(rng, (len(lens), H, L, D), dtype).cuda() for _ in range(2))
    k[0, 0, -1, 0] = float("inf")
    want = cache.clone()
    for b, n in enumerate(lens):
        c = L if counts is None else min(max(counts[b], 0), L)
        for i in range(max(L - c, L - n, 0), L):
            at = n - L + i
            want[table[b, at // page], 0, :, at % page] = k[b, :, i]
            want[table[b, at // page], 1, :, at % page] = v[b, :, i]
    if tokens_first:                                                             # [B, L, H, D] storage
        k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
    at, counts = on_device(table, lens, counts)
    api.paged_write(cache, k, v, *at, counts=counts)
    api.poll_status()
    assert torch.equal(cache.view(torch.int16), want.view(torch.int16))


@pytest.mark.gpu
def test_bad_pages_and_lengths():
    rng = np.random.default_rng(5)
    cache, table, ks, vs = fill(rng, [40, 40], 2, 64, 16, "f16")
    good = cache.clone()
    q = draw_rows(rng, (2, 4, 1, 64), "f16").cuda()
    k = draw_rows(rng, (2, 2, 1, 64), "f16").cuda()
    lens = ints([40, 40]).cuda()

    def reported(call):
        got = call()
        with pytest.raises(_lib.SdpaError) as e:
            api.poll_status()
        assert e.value.status == INDEX
        return got

    for bad in (-1, cache.shape[0], 2**31 - 1):
        broken = table.clone()
        broken[0, 1] = bad                                                       # hides tokens 16..31
        out, lse = reported(lambda: api.paged_attention(q, cache, broken.cuda(), lens, need_lse=True))
        cut = [np.delete(x[0], slice(16, 32), 1) for x in (ks, vs)]
        check(out, lse, q, [cut[0], ks[1]], [cut[1], vs[1]], 1 / 8, False, "f16")
        w = torch.zeros(2, 2, 40, device="cuda")
        reported(lambda: api.paged_weights(q, cache, broken.cuda(), lens, lse, w))
        assert not w[0, :, 16:32].any() and (w[0, :, :16] > 0).all() and abs(w.sum().item() - 8) < 1e-4
        broken = table.clone()
        broken[0, 2] = bad
        reported(lambda: api.paged_write(cache, k, k, broken.cuda(), lens, counts=ints([1, 0]).cuda()))
        assert torch.equal(cache.view(torch.int16), good.view(torch.int16))
    # past the table's end, past max_len, below zero
    out, _ = reported(lambda: api.paged_attention(q, cache, table.cuda(), ints([49, 40]).cuda(), is_causal=False, max_len=40))
    check(out, None, q, ks, vs, 1 / 8, False, "f16")
    out, lse = reported(lambda: api.paged_attention(q, cache, table.cuda(), ints([-5, 40]).cuda(), need_lse=True))
    assert not out[0].any() and torch.isneginf(lse[0]).all()
    reported(lambda: api.paged_write(cache, k, k, table.cuda(), ints([49, -1]).cuda()))
    assert torch.equal(cache.view(torch.int16), good.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("scale", [0.1, 0.0, -0.1])
@pytest.mark.parametrize("L", [4, 20, 70, 200])
def test_bad_pages_in_chunks(L, scale, D):
    """Tokens 16..31 and 112..127 lie on pages that do not exist, for attention and weights alike."""
    rng = np.random.default_rng(6)
    n, gone = 260, [*range(16, 32), *range(112, 128)]
    cache, table, ks, vs = fill(rng, [n], 1, D, 16, "bf16")
    q = draw_rows(rng, (1, 4, L, D), "bf16")
    broken = table.clone()
    broken[0, 1], broken[0, 7] = -1, cache.shape[0]
    out, lse = api.paged_attention(q.cuda(), cache, broken.cuda(), ints([n]).cuda(), need_lse=True, scale=scale)
    with pytest.raises(_lib.SdpaError) as e:
        api.poll_status()
    assert e.value.status == INDEX
    # Query i sees the tokens that are there up to its own; those before the first query lie before all rows.
    kept = np.delete(np.arange(n), gone)
    assert n - L >= 128 or L == 200
    if L <= 130:
        check(out, lse, q, [np.delete(ks[0], gone, 1)], [np.delete(vs[0], gone, 1)], scale, True, "bf16")
    else:
        late = kept[kept >= n - L].size                                          # rows of whose own tokens are there
        rows = np.searchsorted(np.arange(n - L, n), kept[kept >= n - L])
        check(out[:, :, rows], lse[:, :, rows].contiguous(), q[:, :, rows], [ks[0][:, kept]], [vs[0][:, kept]], scale, True, "bf16", few=False)
        assert late == rows.size
    w = torch.zeros(1, 1, n, device="cuda")
    api.paged_weights(q.cuda(), cache, broken.cuda(), ints([n]).cuda(), lse, w, scale=scale)
    with pytest.raises(_lib.SdpaError):
        api.poll_status()
    assert not w[0, 0, gone].any() and abs(w.sum().item() - 4 * L) < 1e-2


@pytest.mark.gpu
@pytest.mark.parametrize("G,L,D", [(4, 60, 64), (4, 300, 128), (2, 40, 256), (4, 8, 64), (4, 1, 128)])
def test_nan_values_cost_little(G, L, D):
    """A cache whose values are NaN throughout takes no more than 100 times as long (it is not
    summed anew by hand), and everything that sees one is NaN."""
    rng = np.random.default_rng(34)
    n = 6000
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

    _, plain = timed()
    cache[:, 1] = NAN
    out, slow = timed()
    api.poll_status()
    assert out.isnan().all() and slow < 100 * max(plain, 0.05)


CASES = [
    # dtype, Hq, Hkv, L, D, page, lens, counts
    ("bf16", 1, 1, 1, 64, 16, [1], None),
    ("f16", 4, 4, 1, 32, 16, [15, 16, 17, 0], None),
    ("bf16", 8, 2, 1, 128, 16, [33, 1, 250], None),
    ("f16", 7, 1, 1, 96, 48, [100, 47, 48, 49], None),
    ("bf16", 4, 1, 1, 256, 64, [129, 64], None),
    ("f16", 16, 2, 2, 128, 16, [2, 1, 65, 127], [2, 2, 1, 0]),
    ("bf16", 8, 2, 8, 128, 64, [200, 8, 3, 0], None),              # 32 rows a head
    ("bf16", 6, 2, 5, 96, 32, [77, 32, 4], [5, 3, 5]),
    ("f16", 8, 2, 3, 32, 16, [500, 31], None),
    ("f16", 4, 2, 6, 256, 16, [90, 6], None),
    ("bf16", 32, 8, 1, 128, 64, [1500, 700, 1029, 64], None),
    ("f16", 12, 3, 1, 64, 112, [3333], None),
    ("bf16", 4, 1, 11, 128, 16, [40, 70], None),                   # more rows than one warp tile's
    ("f16", 3, 3, 40, 64, 16, [64, 39], [40, 12]),
    ("bf16", 4, 2, 130, 128, 16, [130, 300], None),
    ("f16", 9, 3, 61, 96, 48, [61, 150, 200], [61, 20, 0]),        # 183 rows of three heads
    ("bf16", 5, 1, 100, 32, 32, [100, 129], None),
    ("f16", 2, 2, 257, 64, 80, [257, 400], None),
    ("bf16", 2, 1, 200, 256, 48, [200, 333], [200, 77]),
    ("bf16", 48, 1, 9, 64, 16, [9, 140], None),                    # 48 query heads a KV head
    ("f16", 160, 1, 3, 64, 16, [50, 3], None),                     # more query heads than a tile has rows
    ("bf16", 131, 1, 2, 32, 32, [70], None),                       # a prime number of them
    ("bf16", 64, 1, 1, 128, 16, [200, 1], None),
    ("f16", 17, 1, 1, 96, 16, [140, 0], None),
    ("bf16", 4, 1, 10, 32, 16, [150, 10], None),                   # one tile of rows at every head dim
    ("f16", 3, 1, 20, 96, 48, [170, 30], [20, 7]),
    ("bf16", 8, 2, 25, 128, 64, [25, 190], None),
    ("f16", 2, 1, 33, 256, 16, [133, 35], [33, 1]),
    ("f16", 4, 2, 50, 32, 65536, [300, 50], None),                 # the largest pages
    ("bf16", 2, 2, 1, 64, 65536, [77], None),
]


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("dtype,Hq,Hkv,L,D,page,lens,counts", CASES)
def test_attention(dtype, Hq, Hkv, L, D, page, lens, counts, sinks, causal):
    rng = np.random.default_rng(1000 * L + D + len(lens))
    cache, table, ks, vs = fill(rng, lens, Hkv, D, page, dtype)
    q = draw_rows(rng, (len(lens), Hq, L, D), dtype, 1.5)
    sink = None
    if sinks:
        sink = rng.standard_normal(Hq).astype(np.float32) + 2
        sink[0] = 30.0 if Hq > 1 else sink[0]
        sink[-1] = -np.inf if Hq > 2 else sink[-1]
    at, dev_counts = on_device(table, lens, counts)
    how = dict(is_causal="bottom_right" if causal else False, sinks=None if sink is None else torch.from_numpy(sink).cuda(), counts=dev_counts)
    out, lse = api.paged_attention(q.cuda(), cache, *at, need_lse=True, **how)
    again, none = api.paged_attention(q.cuda(), cache, *at, max_len=max(lens), **how)
    api.poll_status()
    assert none is None
    scale = 1 / math.sqrt(D)
    check(out, lse, q, ks, vs, scale, causal, dtype, counts, sink)
    check(again, None, q, ks, vs, scale, causal, dtype, counts, sink)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
@pytest.mark.parametrize("L", [1, 60])
def test_scales(dtype, scale, L):
    rng = np.random.default_rng(17)
    cache, table, ks, vs = fill(rng, [150, 61], 2, 64, 16, dtype)
    q = draw_rows(rng, (2, 4, L, 64), dtype)
    out, lse = api.paged_attention(q.cuda(), cache, table.cuda(), ints([150, 61]).cuda(), scale=scale, need_lse=True)
    api.poll_status()
    check(out, lse, q, ks, vs, scale, True, dtype)


ROWS = [(128, 4, 1), (128, 4, 6), (64, 2, 40), (96, 3, 150), (256, 1, 1), (256, 2, 70), (32, 8, 33)]  # D, G, L


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,G,L", ROWS)
@pytest.mark.parametrize("what", [NAN, float("inf"), -float("inf")])
def test_what_is_hidden_leaves_no_trace(D, G, L, dtype, what):
    """Tokens after a row's own, in this call's rows and on the page behind them, and rows of q
    that are padding."""
    rng = np.random.default_rng(31)
    lens = [L + 60, L, L + 131]
    cache, table, ks, vs = fill(rng, lens, 2, D, 32, dtype)
    q = draw_rows(rng, (3, 2 * G, L, D), dtype)
    at, _ = on_device(table, lens)
    out, lse = api.paged_attention(q.cuda(), cache, *at, need_lse=True)
    # Spoil the last token: only the last row may notice.
    for b, n in enumerate(lens):
        cache[table[b, (n - 1) // 32], :, :, (n - 1) % 32] = what
    got, got_lse = api.paged_attention(q.cuda(), cache, *at, need_lse=True)
    api.poll_status()
    if L > 1:
        assert torch.equal(got[:, :, :-1], out[:, :, :-1]) or (got[:, :, :-1].float() - out[:, :, :-1].float()).abs().max() < 0.02
        check(got[:, :, :-1].contiguous(), got_lse[:, :, :-1].contiguous(), q[:, :, :-1], [k[:, :-1] for k in ks], [v[:, :-1] for v in vs],
              1 / math.sqrt(D), True, dtype, few=G * L <= 32)
    if math.isnan(what):
        assert got[:, :, -1].isnan().all() and got_lse[:, :, -1].isnan().all()
    if L > 1:
        q[:, :, 0] = what
        counts = ints([L - 1] * 3).cuda()
        got, got_lse = api.paged_attention(q.cuda(), cache, *at, need_lse=True, counts=counts)
        api.poll_status()
        assert not got[:, :, 0].any() and torch.isneginf(got_lse[:, :, 0]).all()
        assert got[:, :, 1:-1].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,G,L", ROWS)
def test_a_value_that_is_not_finite_reaches_the_rows_that_see_it(D, G, L, dtype):
    """A NaN in one element of one value and an infinity in another's: their columns, from the
    first row that sees them on, and nothing else."""
    rng = np.random.default_rng(32)
    n = L + 45
    cache, table, ks, vs = fill(rng, [n], 1, D, 16, dtype)
    q = draw_rows(rng, (1, G, L, D), dtype, 0.3)
    j, k = n - 1 - L // 3, n - 1 - L // 2                                         # in the call's own rows
    cache[table[0, j // 16], 1, 0, j % 16, 5] = NAN
    cache[table[0, k // 16], 1, 0, k % 16, D - 3] = -float("inf")
    out, lse = api.paged_attention(q.cuda(), cache, table.cuda(), ints([n]).cuda(), need_lse=True)
    api.poll_status()
    pos = n - L + np.arange(L)
    got = as_f64(out)[0]
    assert np.isnan(got[:, pos >= j, 5]).all() and np.isneginf(got[:, pos >= k, D - 3]).all()
    vs[0][0, j, 5] = vs[0][0, k, D - 3] = 0
    rest = torch.from_numpy(got.copy())
    rest[:, pos >= j, 5] = 0
    rest[:, pos >= k, D - 3] = 0
    o = ref.attention(as_f64(q), ks, vs, 1 / math.sqrt(D), True)[0][0]
    o[:, pos >= j, 5] = o[:, pos >= k, D - 3] = 0
    assert rest.isfinite().all() and np.abs(rest.numpy() - o).max() < 0.03 and torch.isfinite(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("D,G,L", ROWS)
def test_a_nan_key_reaches_out_and_lse(D, G, L):
    rng = np.random.default_rng(33)
    for at in (0, 5, 100):
        n = L + 120
        cache, table, _, _ = fill(rng, [n], 1, D, 16, "bf16")
        cache[table[0, at // 16], 0, 0, at % 16, 1] = NAN
        q = draw_rows(rng, (1, G, L, D), "bf16")
        out, lse = api.paged_attention(q.cuda(), cache, table.cuda(), ints([n]).cuda(), need_lse=True)
        api.poll_status()
        assert out.isnan().all() and lse.isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,G,L,D", [("bf16", 4, 1, 128), ("f16", 2, 8, 64), ("bf16", 1, 1, 256), ("f16", 4, 40, 96), ("bf16", 4, 70, 128), ("bf16", 2, 70, 256)])
def test_sequences_of_several_chunks(dtype, G, L, D):
    rng = np.random.default_rng(41)
    lens = [9000, max(L, 513), 2049]
    cache, table, ks, vs = fill(rng, lens, 1, D, 64, dtype)
    q = draw_rows(rng, (3, G, L, D), dtype)
    at, _ = on_device(table, lens)
    need = _lib.sdpa_paged_attn_workspace_size(api._paged(cache, *at, 3), 3, G, L, 0)
    assert need > 0                                                              # they are cut
    out, lse = api.paged_attention(q.cuda(), cache, *at, need_lse=True)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")              # its contents do not matter
    again, _ = api.paged_attention(q.cuda(), cache, *at, workspace=ws)
    api.poll_status()
    assert torch.equal(out, again)
    check(out, lse, q, ks, vs, 1 / math.sqrt(D), True, dtype)
    with pytest.raises(_lib.SdpaError) as e:
        api.paged_attention(q.cuda(), cache, *at, workspace=ws[:need - 16])
    assert e.value.status == WORKSPACE


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,L,n,D", [(4, 1, 10240, 10240, 32), (8, 2, 5200, 5300, 64), (32, 8, 1500, 9000, 128), (2, 1, 3000, 20000, 256)])
def test_long_chunks_agree_with_the_dense_kernel(Hq, Hkv, L, n, D, causal):
    """Whole waves of blocks and what is left over of them, at sizes that are too large for the oracle.
    Both kernels' outputs lie within half·|o| + half·A of the exact ones (paged_util.check), A at most
    sqrt(sum w^2)-fold less than max|v| here: values are N(0, 1), outputs of n >= 1000 visible tokens
    below 0.5 and A below 1; rows that see fewer tokens are left to the other tests."""
    rng = np.random.default_rng(42)
    cache, table, _, _ = fill(rng, [n], Hkv, D, 64, "bf16")
    rows = cache[table[0].long().cuda()].permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :n].unsqueeze(1)
    q = draw_rows(rng, (1, Hq, L, D), "bf16").cuda()
    out, lse = api.paged_attention(q, cache, table.cuda(), ints([n]).cuda(), need_lse=True, is_causal="bottom_right" if causal else False)
    want, want_lse = api.attention_forward(q, rows[0].contiguous(), rows[1].contiguous(), is_causal="bottom_right" if causal else False)
    api.poll_status()
    first = max(0, 1000 - (n - L))
    half = 2.0**-9
    assert (out - want)[:, :, first:].float().abs().max() <= 2 * half * (0.5 + 1.0)
    assert (lse - want_lse).abs().max() <= 2.0**-15


@pytest.mark.gpu
@pytest.mark.parametrize("L", [2, 50])
def test_layouts_and_another_stream(L):
    rng = np.random.default_rng(43)
    lens = [90, 70]
    cache, table, ks, vs = fill(rng, lens, 2, 64, 32, "f16")
    wide = draw_rows(rng, (2, L, 3, 6, 64), "f16").cuda()
    q = wide[:, :, 1].transpose(1, 2)                                            # [2, 6, L, 64] of a fused projection
    out = torch.zeros(2, L, 6, 64, dtype=torch.float16, device="cuda").transpose(1, 2)
    at, _ = on_device(torch.cat([table, table], 1)[:, :table.shape[1]], lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, lse = api.paged_attention(q, cache, *at, out=out, need_lse=True, stream=side)
    api.poll_status(side)
    assert got is out
    check(out, lse, q, ks, vs, 1 / 8, True, "f16")


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """The last page of a cache of more than 4 GiB (and 2^31 elements)."""
    pages, H, page, D = 2100, 4, 1024, 128
    cache = torch.empty((pages, 2, H, page, D), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(7)
    k, v = (draw_rows(rng, (1, H, 20, D), "bf16").cuda() for _ in range(2))
    table = ints([[pages - 1]]).cuda()
    api.paged_write(cache, k, v, table, ints([20]).cuda())
    for L in (1, 20):
        q = draw_rows(rng, (1, 4 * H, L, D), "bf16")
        out, lse = api.paged_attention(q.cuda(), cache, table, ints([20]).cuda(), need_lse=True)
        api.poll_status()
        check(out, lse, q, [as_f64(k)[0]], [as_f64(v)[0]], D**-0.5, True, "bf16")


@pytest.mark.gpu
def test_python_refusals():
    cache = api.paged_empty(4, 2, 16, 64, torch.float16)
    q = torch.zeros(2, 4, 3, 64, dtype=torch.float16, device="cuda")
    k = q[:, :2]
    table, lens = ints([[0], [1]]).cuda(), ints([3, 3]).cuda()
    for bad in (lambda: api.paged_write(cache, k.bfloat16(), k, table, lens), lambda: api.paged_write(cache, k, k[:, :1], table, lens),
                lambda: api.paged_write(cache, q, q, table, lens), lambda: api.paged_write(cache, k, k, table.long(), lens),
                lambda: api.paged_write(cache, k, k, table[:1], lens), lambda: api.paged_write(cache, k, k, table, lens.long()),
                lambda: api.paged_write(cache, k, k, table, lens, counts=lens[:1]), lambda: api.paged_write(cache[:, :, :, :8], k, k, table, lens),
                lambda: api.paged_write(cache[0], k, k, table, lens), lambda: api.paged_attention(q[..., :32], cache, table, lens),
                lambda: api.paged_attention(q[0], cache, table, lens), lambda: api.paged_attention(q, cache, table, lens, is_causal=5),
                lambda: api.paged_attention(q, cache.cpu(), table, lens), lambda: api.paged_attention(q, cache, table.cpu(), lens),
                lambda: api.paged_attention(q, cache, table, lens, sinks=torch.zeros(3, device="cuda")),
                lambda: api.paged_attention(q, cache, table, lens, need_lse=True, lse=torch.zeros(2, 4, 3, device="cuda").half()),
                lambda: api.paged_attention(q, cache, table, lens, out=q[:, :2]),
                lambda: api.paged_attention(q, cache, table, lens, workspace=torch.zeros(9, 9, device="cuda")[:, :5])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(_lib.SdpaError):
        api.paged_attention(q, cache, table, lens, is_causal=True)
    with pytest.raises(_lib.SdpaError):
        api.paged_attention(q, cache, table, lens, out=q)
    with pytest.raises(_lib.SdpaError):
        api.paged_attention(q[:, :3], cache, table, lens)


@pytest.mark.gpu
def test_two_graphs_on_their_own_workspaces():
    """Two captured calls of different lengths, replayed in turn and on two streams at once."""
    rng = np.random.default_rng(47)
    runs = []
    for n, L in ((5000, 1), (3000, 40)):
        cache, table, ks, vs = fill(rng, [n], 2, 64, 64, "bf16")
        q = draw_rows(rng, (1, 8, L, 64), "bf16").cuda()
        at, _ = on_device(table, [n])
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            api.paged_attention(q, cache, *at)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out, lse = api.paged_attention(q, cache, *at, need_lse=True)
        runs.append((graph, stream, q, out, lse, ks, vs, cache, at))             # the graph reads cache and at
    for _ in range(3):
        for graph, stream, q, *_ in runs:
            q.copy_(draw_rows(rng, tuple(q.shape), "bf16"))
        torch.cuda.synchronize()
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        api.poll_status()
        for _, _, q, out, lse, ks, vs, *_ in runs:
            check(out, lse, q, ks, vs, 1 / 8, True, "bf16")
