"""The 4-bit paged cache: writing (bytes equal to the oracle's packing) and reading back.

Reading: z + s·c in fp32, rounded once to T: |error| <= (eps(T)/2 + 2^-24)·|value|, and
2^-25 where fp16 has no smaller step.
"""
import numpy as np
import pytest
import torch

from cache_util import TYPES, dirty_cache, draw_rows, held, ints, make_table
from oracle import cache as ref
from scaled_dot_product_flash_gb300 import _lib, api, build
from scaled_dot_product_flash_gb300.inputs import as_f64

INVALID, UNSUPPORTED, INDEX = 1, 2, 6


def check_values(got, want, dtype):
    got, want = as_f64(got), np.asarray(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    want = np.nan_to_num(want)
    tol = (torch.finfo(TYPES[dtype]).eps / 2 + 2.0**-24) * np.abs(want) + (2.0**-25 if dtype == "f16" else 0)
    assert (np.abs(np.nan_to_num(got) - want) <= tol).all(), np.abs(np.nan_to_num(got) - want).max()


# ---- without a GPU


def test_oracle_format():
    """Closed forms: codes at the ends, a tie, a constant group, and a group that is not finite."""
    x = np.zeros((1, 96))
    x[0, :32] = np.arange(32) % 16                       # s = 1: the codes are the elements
    x[0, 32:64] = 2.5
    x[0, 70] = np.inf
    code, s, z = ref.quantise(x, torch.bfloat16)
    assert np.array_equal(code[0, :32], np.arange(32) % 16) and s[0, 0] == 1 and z[0, 0] == 0
    assert s[0, 1] == 0 and z[0, 1] == 2.5 and not code[0, 32:64].any()
    assert np.isnan(z[0, 2]) and s[0, 2] == 0
    y = np.zeros((1, 32))
    y[0, :4] = [0, 30, 5, 7]                             # s = 2: 2.5 and 3.5 round to 2 and 4
    assert ref.quantise(y, torch.float16)[0][0, :4].tolist() == [0, 15, 2, 4]


@pytest.mark.parametrize("D", [32, 64, 96, 128, 256])
def test_oracle_places_fill_the_tile_once(D):
    k, v, p = ref.word_places(D)
    seen = set(k.values()) | set(v.values())
    assert len(seen) == 2 * 16 * D and {b for b, _ in seen} == set(range(16 * D))
    assert sorted(p.values()) == list(range(0, 2 * D, 4))


def test_cache_sizes():
    build.build()
    assert _lib.sdpa_cache_page_bytes(64, 8, 128, 2) == 8 * 4 * 2560
    for bad in ((63, 8, 128, 2), (0, 8, 128, 2), (64, 0, 128, 2), (64, 8, 80, 2), (64, 8, 128, 0), (64, 8, 128, 3), (131072, 8, 128, 2)):
        assert _lib.sdpa_cache_page_bytes(*bad) == 0
    c = api.cache_empty(3, 2, 48, 96, torch.float16, device="cpu")
    assert c.shape == (3, 2, 3, 960) and c.numel() * 2 == 3 * _lib.sdpa_cache_page_bytes(48, 2, 96, 1)
    for bad in (dict(dtype=torch.float32), dict(page_size=40), dict(num_pages=0), dict(head_dim=48)):
        with pytest.raises(ValueError):
            api.cache_empty(**dict(dict(num_pages=3, num_kv_heads=2, page_size=32, head_dim=64, device="cpu"), **bad))


def test_host_tensors_are_refused():
    cache = api.cache_empty(3, 2, 16, 64, device="cpu")
    k = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.cache_write(cache, k, k, ints([[0]]), ints([3]))
    with pytest.raises(ValueError):
        api.cache_read(cache, ints([[0]]), ints([3]), 3)


# Fake, 16-byte aligned addresses: every case is rejected before anything is launched.
DATA, TABLE, LENS, K, V, COUNTS = (0x10000000 * (n + 1) for n in range(6))
GOOD = dict(data=DATA, num_pages=4, page_size=32, Hkv=2, D=64, dtype=2, pages=TABLE, pages_stride=3, pages_per_seq=2, lens=LENS)


def refused_cases():
    return [
        (dict(data=0), INVALID), (dict(data=DATA + 8), INVALID), (dict(pages=0), INVALID), (dict(lens=0), INVALID),
        (dict(pages=TABLE + 2), INVALID), (dict(lens=LENS + 1), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=24), INVALID),
        (dict(page_size=0), INVALID), (dict(Hkv=0), INVALID), (dict(pages_stride=1), INVALID), (dict(pages_per_seq=0), INVALID),
        (dict(D=48), UNSUPPORTED), (dict(dtype=0), UNSUPPORTED), (dict(dtype=5), UNSUPPORTED), (dict(page_size=131072), UNSUPPORTED),
        (dict(page_size=65536, pages_per_seq=32768, pages_stride=32768), UNSUPPORTED),
        (dict(B=0), INVALID), (dict(L=0), INVALID), (dict(B=70000), UNSUPPORTED), (dict(B=60000, L=60000), UNSUPPORTED),
        (dict(k=0), INVALID), (dict(v=V + 2), INVALID), (dict(lay=None), INVALID),
        (dict(lay=(4096, 2048, 64, 4096, 0, 64)), INVALID),         # heads on one address
        (dict(lay=(4096, 2048, 68, 4096, 2048, 64)), INVALID),      # rows off the 16-byte grid
        (dict(k=DATA + 64), INVALID),                               # rows inside the cache
    ]


def call(read, **kw):
    a = dict(GOOD, B=2, L=5, k=K, v=V, counts=None, lay=(4096, 2048, 64, 4096, 2048, 64))
    a.update(kw)
    c = _lib.Cache(*(a[n] for n in GOOD))
    build.build()
    lay = None if a["lay"] is None else _lib.Int64x6(*a["lay"])
    if read:
        return _lib.sdpa_cache_read(c, a["k"], a["v"], lay, a["B"], a["L"], None)
    return _lib.sdpa_cache_write(c, a["k"], a["v"], lay, a["counts"], a["B"], a["L"], None)


@pytest.mark.parametrize("kw,code", refused_cases() + [
    (dict(counts=COUNTS + 2), INVALID), (dict(counts=DATA + 4), INVALID), (dict(lens=DATA), INVALID), (dict(pages=DATA + 16), INVALID)])
def test_write_refused(kw, code):
    assert call(False, **kw) == code


@pytest.mark.parametrize("kw,code", refused_cases() + [
    (dict(v=K), INVALID), (dict(k=TABLE), INVALID), (dict(v=LENS), INVALID)])
def test_read_refused(kw, code):
    assert call(True, **kw) == code


def test_null_cache_refused():
    lib = _lib.load(build.build())
    assert lib.sdpa_cache_write(None, K, V, None, None, 1, 1, None) == INVALID
    assert lib.sdpa_cache_read(None, K, V, None, 1, 1, None) == INVALID


# ---- on the GPU


def expected(cache, rows, table, lens, counts, page, dtype):
    """The bytes of `cache` (uint8 numpy, in place) after the oracle wrote the rows."""
    k, v = (as_f64(x) for x in rows)
    B, H, L, D = k.shape
    places = ref.word_places(D)
    for b in range(B):
        for i in range(max(L - counts[b], L - lens[b], 0), L):
            pos = lens[b] - L + i
            for h in range(H):
                tile = cache[table[b, pos // page], h, pos % page // 16]
                ref.put_token(tile, pos % 16, places, k[b, h, i], v[b, h, i], TYPES[dtype])
    return cache


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,H,L,D,page,lens,counts", [
    ("bf16", 1, 1, 32, 16, [1], None),
    ("bf16", 2, 1, 128, 16, [1, 16, 17, 100], None),
    ("f16", 3, 21, 96, 48, [21, 50, 5, 0], [21, 2, 21, 21]),       # padding, a short sequence, an empty one
    ("f16", 1, 40, 64, 32, [40, 47, 64], [0, 40, 17]),
    ("bf16", 2, 7, 256, 16, [7, 9, 33], [7, 8, 1]),                # a count above the rows
    ("bf16", 2, 35, 128, 64, [100, 36], None),
])
def test_write_and_read(dtype, H, L, D, page, lens, counts):
    rng = np.random.default_rng(D + L)
    table, pages = make_table(rng, lens, page)
    cache = dirty_cache(pages, H, page, D, dtype)
    k, v = (draw_rows(rng, (len(lens), H, L, D), dtype, 3.0) for _ in range(2))
    v[0, 0, -1, :32] = 1.75                                          # a constant group
    k[-1, -1, -1, -1] = float("inf")                                 # a group that is not finite
    before = cache.view(torch.uint8).cpu().numpy().copy()
    api.cache_write(cache, k.cuda(), v.cuda(), table.cuda(), ints(lens).cuda(), None if counts is None else ints(counts).cuda())
    api.poll_status()
    counts = [L] * len(lens) if counts is None else counts
    want = expected(before, (k, v), table.numpy(), lens, counts, page, dtype)
    got = cache.view(torch.uint8).cpu().numpy()
    # NaNs may differ in their bits: compare those as values.
    where = want != got
    if where.any():
        a, b = (torch.from_numpy(x).view(TYPES[dtype]) for x in (want, got))
        assert (torch.isnan(a) & torch.isnan(b))[torch.from_numpy(where).view(torch.int16).view(a.shape) != 0].all()
    # The last rows of every sequence, more of them than were written (0 before position 0).
    # Rows that were never written hold the filling: NaN.
    rows = L + 3
    ko, vo = api.cache_read(cache, table.cuda(), ints(lens).cuda(), rows)
    api.poll_status()
    for x, out in ((k, ko), (v, vo)):
        full = np.full((len(lens), H, rows, D), np.nan)
        for b, n in enumerate(lens):
            full[b, :, :max(0, rows - n)] = 0
            real = min(counts[b], L, n)
            full[b, :, rows - real:] = held(as_f64(x)[b, :, L - real:], dtype)
        check_values(out, full, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_extreme_groups(dtype):
    """The type's largest and smallest values, subnormal scales and wide ranges: bytes equal."""
    top, tiny = torch.finfo(TYPES[dtype]).max, torch.finfo(TYPES[dtype]).smallest_normal
    rng = np.random.default_rng(3)
    x = torch.zeros(1, 1, 8, 64, dtype=torch.float64)
    x[0, 0, 0] = torch.from_numpy(rng.uniform(-1, 1, 64)) * top      # for bf16 the range overflows fp32
    x[0, 0, 1] = torch.from_numpy(rng.uniform(0, 1, 64)) * top
    x[0, 0, 2] = torch.from_numpy(rng.uniform(-1, 1, 64)) * tiny
    x[0, 0, 3] = torch.from_numpy(rng.uniform(-1, 1, 64)) * tiny / 64
    x[0, 0, 4] = 1.0 + torch.from_numpy(rng.uniform(0, 1, 64)) / 64
    x[0, 0, 5, 7] = tiny / 128
    x[0, 0, 6] = -0.0
    x[0, 0, 7] = torch.arange(64) / 8                                # ties
    x = x.to(TYPES[dtype])
    cache = dirty_cache(1, 1, 16, 64, dtype)
    table, lens = ints([[0]]).cuda(), ints([8]).cuda()
    api.cache_write(cache, x.cuda(), x.cuda(), table, lens)
    k, v = api.cache_read(cache, table, lens, 8)
    api.poll_status()
    want = held(as_f64(x), dtype)
    check_values(k, want, dtype)
    check_values(v, want, dtype)


@pytest.mark.gpu
def test_strided_rows_and_another_stream():
    rng = np.random.default_rng(4)
    B, H, L, D = 2, 2, 19, 128
    fused = draw_rows(rng, (B, L, 3, H, D), "bf16").cuda()
    k, v = fused[:, :, 1].transpose(1, 2), fused[:, :, 2].transpose(1, 2)
    table, lens = ints([[1, 3, 0], [2, 4, 0]]).cuda()[:, :2], ints([19, 20]).cuda()   # a table with a longer stride
    one, two = dirty_cache(5, H, 16, D, "bf16"), dirty_cache(5, H, 16, D, "bf16")
    api.cache_write(one, k.contiguous(), v.contiguous(), table, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    api.cache_write(two, k, v, table, lens, stream=side)
    out = api.cache_read(two, table, lens, L, k=torch.empty(B, L, H, D, dtype=k.dtype, device="cuda").transpose(1, 2), stream=side)
    side.synchronize()
    want = api.cache_read(one, table, lens, L)
    api.poll_status()
    assert torch.equal(one.view(torch.uint8), two.view(torch.uint8))
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@pytest.mark.gpu
def test_bad_pages_and_lengths_are_reported():
    """Nothing outside the cache is touched: tokens on bad pages are skipped, read as 0."""
    rng = np.random.default_rng(11)
    H, L, D, page = 2, 20, 64, 16
    whole = dirty_cache(6, H, page, D, "f16")
    cache = whole[1:5]                                                  # pages before and after it stay as they are
    k, v = (draw_rows(rng, (4, H, L, D), "f16") for _ in range(2))
    table = ints([[0, -1], [4, 1], [2, 3], [2, 3]]).cuda()             # -1 and 4 are outside of 0..3
    lens = ints([20, 20, -5, 40]).cuda()                               # a negative length, one past the table's end (32)
    api.cache_write(cache, k.cuda(), v.cuda(), table, lens)
    with pytest.raises(_lib.SdpaError) as e:
        api.poll_status()
    assert e.value.status == INDEX
    assert (whole[0].view(torch.uint8) == 255).all() and (whole[5].view(torch.uint8) == 255).all()
    ko, _ = api.cache_read(cache, table, lens, L)
    with pytest.raises(_lib.SdpaError):
        api.poll_status()
    want = held(as_f64(k), "f16")
    full = np.zeros_like(want)
    full[0, :, :16], full[1, :, 16:] = want[0, :, :16], want[1, :, 16:]
    full[3] = want[3]                                                   # 40 is read as 32: rows are positions 12..31
    check_values(ko, full, "f16")
    api.poll_status()


@pytest.mark.gpu
def test_python_refusals():
    cache = api.cache_empty(4, 2, 16, 64, torch.float16)
    k = torch.zeros(2, 2, 3, 64, dtype=torch.float16, device="cuda")
    table, lens = ints([[0], [1]]).cuda(), ints([3, 3]).cuda()
    bad = [
        (cache, k.bfloat16(), k, table, lens, None), (cache, k[:, :1], k, table, lens, None), (cache, k, k[:, :, :2], table, lens, None),
        (cache, k[..., :32], k, table, lens, None), (cache, k, k, table.long(), lens, None), (cache, k, k, table[0], lens, None),
        (cache, k, k, table[:1], lens, None), (cache, k, k, table, lens.long(), None), (cache, k, k, table, lens[:1], None),
        (cache, k, k, table, lens, lens.long()), (cache, k, k, table, lens, lens[:1]), (cache.float(), k.float(), k.float(), table, lens, None),
        (cache[..., :635], k, k, table, lens, None), (cache, k, k, table.cpu(), lens, None),
    ]
    for args in bad:
        with pytest.raises(ValueError):
            api.cache_write(*args)
    with pytest.raises(ValueError):
        api.cache_read(cache, table, lens, 3, k=k[:, :, :2])
    with pytest.raises(_lib.SdpaError):
        api.cache_read(cache, table, lens, 0)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """The last pages of a cache of more than 2^32 bytes."""
    H, D, page = 8, 128, 128
    pages = (2**32 + 2**28) // _lib.sdpa_cache_page_bytes(page, H, D, 2) + 1
    cache = api.cache_empty(pages, H, page, D)
    rng = np.random.default_rng(12)
    k, v = (draw_rows(rng, (1, H, 5, D), "bf16") for _ in range(2))
    table, lens = ints([[0, pages - 1]]).cuda(), ints([131]).cuda()
    cache[0].zero_()
    api.cache_write(cache, k.cuda(), v.cuda(), table, lens)
    ko, vo = api.cache_read(cache, table, lens, 5)
    api.poll_status()
    check_values(ko, held(as_f64(k), "bf16"), "bf16")
    check_values(vo, held(as_f64(v), "bf16"), "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("L,lens,counts", [
    (1, [33, 32, 2**31 - 1], None),                    # one step too long, the last step there is, far too long
    (3, [35, 32, 40], None), (8, [33, 30, 34], [1, 2, 2]),
])
def test_a_loop_that_runs_too_long_loses_nothing(L, lens, counts):
    """Rows whose positions all lie past the table's end (32 tokens) are not written over the last
    tokens; the second sequence of the batch, which ends in time, is written."""
    rng = np.random.default_rng(14)
    H, D, page = 2, 64, 16
    table = ints([[0, 3], [1, 4], [2, 5]]).cuda()
    cache = dirty_cache(6, H, page, D, "bf16")
    k, v = (draw_rows(rng, (3, H, 32, D), "bf16").cuda() for _ in range(2))
    api.cache_write(cache, k, v, table, ints([32] * 3).cuda())
    api.poll_status()
    before = cache.clone()
    new = [draw_rows(rng, (3, H, L, D), "bf16").cuda() for _ in range(2)]
    counts = None if counts is None else ints(counts).cuda()
    api.cache_write(cache, *new, table, ints(lens).cuda(), counts)
    with pytest.raises(_lib.SdpaError) as e:
        api.poll_status()
    assert e.value.status == INDEX
    api.cache_write(before, *(x[1:2] for x in new), table[1:2], ints(lens[1:2]).cuda(), None if counts is None else counts[1:2])
    api.poll_status()
    assert torch.equal(cache.view(torch.uint8), before.view(torch.uint8))
