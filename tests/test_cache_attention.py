"""Attention over the 4-bit paged cache against the fp64 oracle on the values that the cache
holds, and the cache, the rotary embedding and the attention as they are used together.

Tolerances.  A row's output is sum_j w_j·v_j with v = z + s·c, T the element type:
    eps(T)/2·|o|                  its rounding (2^-25 where fp16 has no smaller step)
  + 2^-11·sum_j w_j·s·c           the products w·s enter the MMA rounded to fp16, the z term
                                  stays in fp32
  + 2^-16·max|v|                  the scores: D products and D/32 scalings summed in fp32, with
                                  |S| up to about 20 off by some 20·2^-22, which moves each
                                  weight by as much relative to itself, twice with the sum
lse: 2^-16·max(1, |lse|), the scores' error and one logarithm.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from cache_util import TYPES, dirty_cache, draw_rows, held, ints, make_table
from oracle import cache as ref
from scaled_dot_product_flash_gb300 import _lib, api, autograd, build
from scaled_dot_product_flash_gb300.inputs import as_f64

INVALID, UNSUPPORTED, WORKSPACE, INDEX = 1, 2, 5, 6


def fill(rng, lens, H, D, page, dtype, width=None, spread=1.0):
    """A cache holding random keys and values of the lengths given, its table, and per sequence
    the fp64 keys and values it holds."""
    table, pages = make_table(rng, lens, page, width)
    cache = dirty_cache(pages, H, page, D, dtype)
    L = max(max(lens), 1)
    k, v = (draw_rows(rng, (len(lens), H, L, D), dtype, spread) for _ in range(2))
    k += torch.from_numpy(rng.standard_normal((1, H, 1, D))).to(k.dtype)     # channels off zero
    api.cache_write(cache, k.cuda(), v.cuda(), table.cuda(), ints(lens).cuda())
    api.poll_status()
    ks, vs, low = [], [], []
    for b, n in enumerate(lens):
        ks.append(held(as_f64(k)[b, :, L - n:], dtype))
        code, s, z = ref.quantise(as_f64(v)[b, :, L - n:], TYPES[dtype])
        vs.append(ref.values(code, s, z))
        low.append(ref.values(code, s, np.zeros_like(z)))                     # s·c alone
    return cache, table, ks, vs, low


def check(out, lse, q, ks, vs, low, scale, causal, sinks, dtype, rows=None):
    o, want_lse = ref.cached_attention(as_f64(q), ks, vs, scale, causal, sinks)
    part, _ = ref.cached_attention(as_f64(q), ks, low, scale, causal, sinks)
    B, Hq = o.shape[:2]
    top = np.zeros((B, Hq, 1, 1))
    for b in range(B):
        if vs[b].size:
            top[b, :, 0, 0] = np.repeat(np.abs(vs[b]).max((1, 2)), Hq // vs[b].shape[0])
    tol = torch.finfo(TYPES[dtype]).eps / 2 * np.abs(o) + 2.0**-11 * part + 2.0**-16 * top + (2.0**-25 if dtype == "f16" else 0)
    got = as_f64(out)
    worst = (np.abs(got - o) / np.maximum(tol, 1e-300)).max()
    assert np.isfinite(got).all() and worst <= 1, f"out is {worst:.2f} of its tolerance"
    if lse is not None:
        got = as_f64(lse)
        none = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got), none)
        off = np.abs(np.where(none, 0, got) - np.where(none, 0, want_lse)) / np.maximum(1, np.abs(np.where(none, 0, want_lse)))
        assert off.max() <= 2.0**-16, f"lse off by {off.max():.2e}"


# ---- without a GPU

DATA, TABLE, LENS, Q, OUT, LSE, SINKS, WS = (0x10000000 * (n + 1) for n in range(8))
GOOD = dict(data=DATA, num_pages=4, page_size=32, Hkv=2, D=64, dtype=2, pages=TABLE, pages_stride=300, pages_per_seq=300, lens=LENS)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), INVALID), (dict(out=0), INVALID), (dict(q=Q + 8), INVALID), (dict(lse=LSE + 4), INVALID), (dict(sinks=SINKS + 2), INVALID),
    (dict(lay=None), INVALID), (dict(lay=(256, 64, 60, 256, 64, 64)), INVALID), (dict(lay=(0, 64, 64, 256, 64, 64)), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID), (dict(causal=3), INVALID), (dict(causal=-1), INVALID),
    (dict(causal=1), UNSUPPORTED), (dict(Hq=3), INVALID), (dict(Hq=0), INVALID), (dict(B=0), INVALID), (dict(Lq=0), INVALID),
    (dict(B=65536), UNSUPPORTED), (dict(Hq=70000), UNSUPPORTED), (dict(dtype=0), UNSUPPORTED), (dict(D=80), UNSUPPORTED),
    (dict(page_size=20), INVALID), (dict(pages_stride=2), INVALID), (dict(data=0), INVALID),
    (dict(out=Q), INVALID), (dict(lse=OUT), INVALID), (dict(out=DATA), INVALID), (dict(out=SINKS - 16), INVALID), (dict(lse=TABLE), INVALID),
    (dict(out=LENS), INVALID),
])
def test_refused(kw, code):
    a = dict(GOOD, q=Q, out=OUT, lse=LSE, sinks=SINKS, lay=(256, 64, 64, 256, 64, 64), B=2, Hq=4, Lq=1, scale=0.125, causal=2, ws=WS, ws_bytes=1 << 26)
    a.update(kw)
    build.build()
    c = _lib.Cache(*(a[n] for n in GOOD))
    lay = None if a["lay"] is None else _lib.Int64x6(*a["lay"])
    assert _lib.sdpa_cache_attn(c, a["q"], a["out"], a["lse"], a["sinks"], lay, a["B"], a["Hq"], a["Lq"], a["scale"], a["causal"], 0, a["ws"],
                                a["ws_bytes"], None) == code


def test_oracle_rows_that_see_nothing():
    q = np.ones((1, 2, 3, 32))
    empty = [np.zeros((1, 0, 32))]
    o, lse = ref.cached_attention(q, empty, empty, 0.1, True)
    assert not o.any() and np.isneginf(lse).all()
    one = [np.full((1, 1, 32), 2.0)]
    o, lse = ref.cached_attention(q, one, one, 0.1, True, np.array([0.5, -np.inf]))
    assert not o[:, :, :2].any() and (lse[0, 0, :2] == 0.5).all() and np.isneginf(lse[0, 1, :2]).all()
    assert np.allclose(o[0, 1, 2], 2.0) and np.allclose(lse[0, 1, 2], 6.4)


# ---- on the GPU

CASES = [
    # dtype, Hq, Hkv, L, D, page, lens
    ("bf16", 1, 1, 1, 64, 16, [1]),
    ("f16", 4, 4, 1, 32, 16, [15, 16, 17, 0]),
    ("bf16", 8, 2, 1, 128, 16, [33, 1, 250]),
    ("f16", 7, 1, 1, 96, 48, [100, 47, 48, 49]),
    ("bf16", 4, 1, 1, 256, 64, [129, 64]),
    ("bf16", 8, 1, 1, 64, 32, [300]),
    ("f16", 16, 2, 2, 128, 16, [2, 1, 65, 127]),          # 16 rows a head, the second before the start
    ("bf16", 8, 2, 8, 128, 64, [200, 8, 3, 0]),           # 32 rows
    ("bf16", 6, 2, 5, 96, 32, [77, 32, 4]),
    ("f16", 8, 2, 3, 32, 16, [500, 31]),
    ("f16", 4, 2, 6, 256, 16, [90, 6]),
    ("bf16", 4, 1, 11, 128, 16, [40, 70]),                # 44 rows a head: more than one block's
    ("f16", 3, 3, 40, 64, 16, [64, 39]),
    ("bf16", 32, 8, 1, 128, 64, [1500, 700, 1029, 64]),
    ("f16", 12, 3, 1, 64, 112, [3333]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("dtype,Hq,Hkv,L,D,page,lens", CASES)
def test_attention(dtype, Hq, Hkv, L, D, page, lens, sinks, causal):
    rng = np.random.default_rng(1000 * L + D + len(lens))
    cache, table, ks, vs, low = fill(rng, lens, Hkv, D, page, dtype)
    q = draw_rows(rng, (len(lens), Hq, L, D), dtype, 1.5)
    sink = None
    if sinks:
        sink = rng.standard_normal(Hq).astype(np.float32) + 2
        sink[0] = 30.0 if Hq > 1 else sink[0]
        sink[-1] = -np.inf if Hq > 2 else sink[-1]
    args = (cache, table.cuda(), ints(lens).cuda())
    how = dict(need_lse=True, is_causal="bottom_right" if causal else False, sinks=None if sink is None else torch.from_numpy(sink).cuda())
    out, lse = api.cache_attention(q.cuda(), *args, **how)
    api.poll_status()
    scale = 1 / math.sqrt(D)
    check(out, lse, q, ks, vs, low, scale, causal, sink, dtype)
    # A tight bound on the lengths gives the same, bit for bit or within the same tolerances.
    out, lse = api.cache_attention(q.cuda(), *args, max_len=max(max(lens), 1), **how)
    api.poll_status()
    check(out, lse, q, ks, vs, low, scale, causal, sink, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(dtype, scale):
    rng = np.random.default_rng(21)
    cache, table, ks, vs, low = fill(rng, [90, 17], 2, 64, 16, dtype)
    q = draw_rows(rng, (2, 4, 2, 64), dtype, 0.4)
    out, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints([90, 17]).cuda(), scale=scale, need_lse=True)
    api.poll_status()
    check(out, lse, q, ks, vs, low, scale, True, None, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,sizes", [("bf16", (1e-20, 1e20)), ("bf16", (1e-3, 1e3)), ("bf16", (1e36, 3e-33)), ("f16", (1e-4, 500.0))])
def test_values_of_any_size(dtype, sizes):
    """Queries and values far from 1, and values whose scale changes by token and by group (the
    keys stay plain, scaled against the queries' size)."""
    rng = np.random.default_rng(22)
    lens, H, D, page = [150], 1, 128, 16
    for size in sizes:
        table, pages = make_table(rng, lens, page)
        cache = dirty_cache(pages, H, page, D, dtype)
        k, v = (draw_rows(rng, (1, H, 150, D), dtype) for _ in range(2))
        v = (v.double() * size * torch.from_numpy(np.exp2(rng.integers(-8, 5, (1, H, 150, 1))))).to(v.dtype)
        v[..., :32] *= 0.03
        q = (draw_rows(rng, (1, 4, 1, D), dtype).double() * size).to(v.dtype)
        api.cache_write(cache, k.cuda(), v.cuda(), table.cuda(), ints(lens).cuda())
        out, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints(lens).cuda(), need_lse=True, scale=0.1 / size)
        api.poll_status()
        code, s, z = ref.quantise(as_f64(v)[0], TYPES[dtype])
        ks, vs, low = [held(as_f64(k)[0], dtype)], [ref.values(code, s, z)], [ref.values(code, s, np.zeros_like(z))]
        check(out, lse, q, ks, vs, low, float(np.float32(0.1 / size)), True, None, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_what_is_hidden_cannot_be_seen(dtype):
    """NaN keys and values at positions behind a query's own leave it alone; the query that sees
    them is NaN.  (The unused places of every cache of these tests are NaN as well.)"""
    rng = np.random.default_rng(23)
    lens, H, L, D, page = [53, 20], 2, 4, 64, 16
    table, pages = make_table(rng, lens, page)
    cache = dirty_cache(pages, H, page, D, dtype)
    k, v = (draw_rows(rng, (2, H, 53, D), dtype) for _ in range(2))
    k[:, :, -1, 5], v[:, :, -2, 40] = float("nan"), float("inf")
    q = draw_rows(rng, (2, 4, L, D), dtype)
    api.cache_write(cache, k.cuda(), v.cuda(), table.cuda(), ints(lens).cuda())
    out, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints(lens).cuda(), need_lse=True)
    api.poll_status()
    assert torch.isnan(out[:, :, 3]).all() and torch.isnan(lse[:, :, 3]).all()
    assert torch.isnan(out[:, :, 2, 32:]).all() and not torch.isnan(out[:, :, 2, :32]).any()
    ks = [held(as_f64(k)[b, :, 53 - n:53 - 2], dtype) for b, n in enumerate(lens)]
    code = [ref.quantise(as_f64(v)[b, :, 53 - n:53 - 2], TYPES[dtype]) for b, n in enumerate(lens)]
    vs = [ref.values(*c) for c in code]
    low = [ref.values(c, s, np.zeros_like(z)) for c, s, z in code]
    check(out[:, :, :2], lse[:, :, :2].contiguous(), q[:, :, :2], ks, vs, low, 1 / 8, True, None, dtype)


@pytest.mark.gpu
def test_a_query_that_is_not_finite_stays_alone():
    rng = np.random.default_rng(24)
    cache, table, ks, vs, low = fill(rng, [70], 1, 128, 16, "bf16")
    q = draw_rows(rng, (1, 8, 1, 128), "bf16")
    clean, _ = api.cache_attention(q.cuda(), cache, table.cuda(), ints([70]).cuda())
    q[0, 3, 0, 17], q[0, 6, 0, 100] = float("nan"), float("inf")
    out, _ = api.cache_attention(q.cuda(), cache, table.cuda(), ints([70]).cuda())
    api.poll_status()
    rows = [0, 1, 2, 4, 5, 7]
    assert torch.equal(out[:, rows], clean[:, rows]) and torch.isnan(out[:, [3, 6]]).all()


@pytest.mark.gpu
def test_bad_pages_and_lengths():
    """Tokens on pages outside the cache are hidden, lengths are cut, both are reported."""
    rng = np.random.default_rng(25)
    lens = [60, 60, 40]
    cache, table, ks, vs, low = fill(rng, lens, 2, 64, 16, "bf16", width=4)
    q = draw_rows(rng, (3, 4, 1, 64), "bf16")
    table[0, 1], table[1, 2] = -1, cache.shape[0]
    out, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints(lens).cuda(), need_lse=True, is_causal=False)
    with pytest.raises(_lib.SdpaError) as e:
        api.poll_status()
    assert e.value.status == INDEX
    gone = {0: (16, 32), 1: (32, 48)}
    for x in (ks, vs, low):
        for b, (lo, hi) in gone.items():
            x[b] = np.concatenate([x[b][:, :lo], x[b][:, hi:]], 1)
    check(out, lse, q, ks, vs, low, 1 / 8, False, None, "bf16")
    # Lengths below 0 and above max_len.
    out, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints([-3, -2**31, 40]).cuda(), need_lse=True, is_causal=False, max_len=24)
    with pytest.raises(_lib.SdpaError):
        api.poll_status()
    none = [np.zeros((2, 0, 64))] * 2
    check(out, lse, q, none + [ks[2][:, :24]], none + [vs[2][:, :24]], none + [low[2][:, :24]], 1 / 8, False, None, "bf16")
    api.poll_status()


@pytest.mark.gpu
def test_layouts_and_another_stream():
    rng = np.random.default_rng(26)
    lens = [100, 37]
    cache, table, *_ = fill(rng, lens, 2, 128, 16, "bf16")
    table, lens = table.cuda(), ints(lens).cuda()
    fused = draw_rows(rng, (2, 3, 12, 128), "bf16").cuda()
    q = fused[:, :, 2:10].transpose(1, 2)                               # [B, H, L, D] out of [B, L, H, D]
    want, want_lse = api.cache_attention(q.contiguous(), cache, table, lens, need_lse=True)
    out = torch.full((2, 3, 12, 128), 7.0, dtype=q.dtype, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, lse = api.cache_attention(q, cache, table, lens, need_lse=True, out=out[:, :, 2:10].transpose(1, 2), stream=side)
    side.synchronize()
    api.poll_status()
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    assert (out[:, :, :2] == 7).all() and (out[:, :, 10:] == 7).all()


@pytest.mark.gpu
def test_long_sequences_and_the_workspace():
    """A length that is split over many blocks, a workspace of the caller's, run-to-run equality,
    and nothing written behind the outputs or the workspace."""
    rng = np.random.default_rng(27)
    lens, Hq, Hkv, D = [9000, 513], 4, 1, 128
    cache, table, ks, vs, low = fill(rng, lens, Hkv, D, 64, "bf16")
    table, dev = table.cuda(), ints(lens).cuda()
    q = draw_rows(rng, (2, Hq, 2, D), "bf16")
    c = api._cache(cache, table, dev, 2)
    need = _lib.sdpa_cache_attn_workspace_size(c, 2, Hq, 2, 0)
    band = torch.full((need + 256,), 113, dtype=torch.uint8, device="cuda")
    outs = torch.full((2 * Hq * 2 * D + 64,), 5.0, dtype=q.dtype, device="cuda")
    out = outs[:2 * Hq * 2 * D].view(2, Hq, 2, D)
    lses = torch.full((2 * Hq * 2 + 16,), 5.0, device="cuda")
    lse = lses[:2 * Hq * 2].view(2, Hq, 2)
    got = api.cache_attention(q.cuda(), cache, table, dev, need_lse=True, out=out, lse=lse, workspace=band[:need])
    api.poll_status()
    check(*got, q, ks, vs, low, 1 / math.sqrt(D), True, None, "bf16")
    assert (band[need:] == 113).all() and (outs[out.numel():] == 5).all() and (lses[lse.numel():] == 5).all()
    again, _ = api.cache_attention(q.cuda(), cache, table, dev)
    assert torch.equal(again, out)
    if need:
        with pytest.raises(_lib.SdpaError) as e:
            api.cache_attention(q.cuda(), cache, table, dev, workspace=band[:need - 16])
        assert e.value.status == WORKSPACE


@pytest.mark.gpu
def test_python_refusals():
    cache = api.cache_empty(4, 2, 16, 64)
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    table, lens = ints([[0]]).cuda(), ints([3]).cuda()
    for kw in (dict(q=q.half()), dict(q=q[..., :32]), dict(q=q[0]), dict(out=q[:, :2]), dict(need_lse=True, lse=torch.zeros(1, 4, 2, device="cuda")),
               dict(sinks=torch.zeros(3, device="cuda")), dict(is_causal=5), dict(pages=table.long()), dict(lens=lens.cpu())):
        with pytest.raises(ValueError):
            api.cache_attention(**dict(dict(q=q, cache=cache, pages=table, lens=lens), **kw))
    with pytest.raises(_lib.SdpaError):
        api.cache_attention(q, cache, table, lens, is_causal=True)
    with pytest.raises(_lib.SdpaError):
        api.cache_attention(q[:, :3], cache, table, lens)


@pytest.mark.gpu
def test_decoding_steps_in_a_graph():
    """Rotary, write and attention of one decoding step, captured once and replayed for several
    steps of a padded batch, against the oracle on everything written so far."""
    rng = np.random.default_rng(28)
    B, Hq, Hkv, D, page, start, steps = 3, 8, 2, 64, 16, [30, 0, 13], 5
    inv = (10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
    dev_inv = torch.from_numpy(inv).cuda()
    width = 3
    table, pages = make_table(rng, [n + steps for n in start], page, width)
    table = table.cuda()
    cache = dirty_cache(pages, Hkv, page, D, "bf16")
    # The prompts: left-padded to 30, rotated by each token's position.
    L = max(start)
    pos = np.array(start)[:, None] - L + np.arange(L)
    k, v = (draw_rows(rng, (B, Hkv, L, D), "bf16") for _ in range(2))
    ko, _ = api.rotary(k.cuda(), None, torch.from_numpy(pos).cuda(), dev_inv)
    api.cache_write(cache, ko, v.cuda(), table, ints(start).cuda())
    ks = [held(as_f64(ko)[b, :, L - n:], "bf16") for b, n in enumerate(start)]
    vq = [ref.quantise(as_f64(v)[b, :, L - n:], torch.bfloat16) for b, n in enumerate(start)]
    vs, low = [ref.values(*x) for x in vq], [ref.values(c, s, np.zeros_like(z)) for c, s, z in vq]
    q1 = torch.zeros(B, Hq, 1, D, dtype=torch.bfloat16, device="cuda")
    k1, v1 = (torch.zeros(B, Hkv, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens = ints(start).cuda()

    def step():
        lens.add_(1)
        q2, k2 = api.rotary(q1, k1, (lens - 1).view(B, 1), dev_inv)
        api.cache_write(cache, k2, v1, table, lens)
        return q2, k2, *api.cache_attention(q2, cache, table, lens, need_lse=True)

    with torch.cuda.stream(torch.cuda.Stream()):                       # a first run, taken back
        step()
        lens.sub_(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q2, k2, out, lse = step()
    for n in range(steps):
        for x in (q1, k1, v1):
            x.copy_(draw_rows(rng, tuple(x.shape), "bf16"))
        graph.replay()
        api.poll_status()
        assert lens.tolist() == [x + n + 1 for x in start]
        position = np.array([[[x + n] for x in start]])
        turned = ref.rotary(as_f64(k1), position, inv)
        assert np.abs(as_f64(k2) - turned).max() <= 2.0**-8 * np.abs(turned).max() + 1e-5
        for b in range(B):
            ks[b] = np.concatenate([ks[b], held(as_f64(k2)[b], "bf16")], 1)
            code, s, z = ref.quantise(as_f64(v1)[b], torch.bfloat16)
            vs[b] = np.concatenate([vs[b], ref.values(code, s, z)], 1)
            low[b] = np.concatenate([low[b], ref.values(code, s, np.zeros_like(z))], 1)
        check(out, lse, q2, ks, vs, low, 1 / 8, True, None, "bf16")


@pytest.mark.gpu
def test_two_graphs_on_their_own_workspaces():
    """Two captured calls replayed at once on two streams give what each gives alone."""
    rng = np.random.default_rng(29)
    lens = [5000]
    cache, table, *_ = fill(rng, lens, 1, 128, 64, "bf16")
    table, dev = table.cuda(), ints(lens).cuda()
    qs = [draw_rows(rng, (1, 4, 1, 128), "bf16").cuda() for _ in range(2)]
    want = [api.cache_attention(q, cache, table, dev)[0] for q in qs]
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(api.cache_attention(q, cache, table, dev)[0])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    api.poll_status()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.gpu
def test_a_chunk_through_the_tiled_kernels():
    """A prompt in two chunks: the second reads the prefix back and runs the tiled attention,
    bottom-right causal, and agrees with the attention over the cache."""
    rng = np.random.default_rng(30)
    H, D, n, L = 2, 128, 200, 72
    cache, table, ks, vs, low = fill(rng, [n], H, D, 16, "bf16")
    q = draw_rows(rng, (1, 2 * H, L, D), "bf16")
    k, v = api.cache_read(cache, table.cuda(), ints([n]).cuda(), n)
    tiled, _ = api.attention_forward(q.cuda(), k, v, is_causal="bottom_right")
    direct, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints([n]).cuda(), need_lse=True)
    api.poll_status()
    check(direct, lse, q, ks, vs, low, 1 / math.sqrt(D), True, None, "bf16")
    o, _ = oracle.sdpa_forward(as_f64(q), as_f64(k), as_f64(v), 1 / math.sqrt(D), 2)
    assert np.abs(as_f64(tiled) - o).max() <= 8e-3


@pytest.mark.gpu
def test_a_training_step():
    """Rotary with two axes, then the attention, differentiated through both."""
    rng = np.random.default_rng(31)
    B, Hq, Hkv, L, D = 1, 4, 2, 50, 64
    q, k, v, g = (torch.from_numpy(rng.standard_normal((B, H, L, D))).float() for H in (Hq, Hkv, Hkv, Hq))
    positions, axes = rng.integers(0, 40, (2, B, L)), np.array([0] * 10 + [1] * 22, dtype=np.int32)
    inv = (100.0 ** (-np.arange(32) / 32)).astype(np.float32)
    leaves = [x.cuda().requires_grad_() for x in (q, k, v)]
    args = (torch.from_numpy(positions).cuda(), torch.from_numpy(inv).cuda(), torch.from_numpy(axes).cuda())
    q2, k2 = autograd.rotary_embedding(leaves[0], leaves[1], *args)
    out = autograd.scaled_dot_product_attention(q2, k2, leaves[2], is_causal=True, enable_gqa=True)
    out.backward(g.cuda())
    api.poll_status()
    qr, kr = (ref.rotary(as_f64(x), positions, inv, axes) for x in (q, k))
    o, _ = oracle.sdpa_forward(qr, kr, as_f64(v), 1 / 8, 1)
    dq, dk, dv = oracle.sdpa_backward(qr, kr, as_f64(v), as_f64(g), 1 / 8, 1)
    dq, dk = (ref.rotary(x, positions, inv, axes, inverse=True) for x in (dq, dk))
    assert np.abs(as_f64(out.detach()) - o).max() <= 1e-5
    for x, want in zip(leaves, (dq, dk, dv)):
        assert np.abs(as_f64(x.grad) - want).max() <= 1e-4


@pytest.mark.gpu
def test_many_short_sequences():
    """More sequences than blocks in a wave, some empty, three rows a KV head."""
    rng = np.random.default_rng(32)
    lens = [int(x) for x in rng.integers(0, 40, 500)]
    cache, table, ks, vs, low = fill(rng, lens, 1, 32, 16, "bf16")
    q = draw_rows(rng, (500, 3, 1, 32), "bf16")
    out, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints(lens).cuda(), need_lse=True)
    api.poll_status()
    check(out, lse, q, ks, vs, low, 1 / math.sqrt(32), True, None, "bf16")


@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls of different shapes on two streams, each with its own memory, as each gives alone."""
    rng = np.random.default_rng(33)
    jobs = []
    for D, lens, H, L in ((128, [4000, 100], 2, 1), (64, [900], 1, 5)):
        cache, table, *_ = fill(rng, lens, H, D, 32, "f16")
        q = draw_rows(rng, (len(lens), 4 * H, L, D), "f16").cuda()
        args = (q, cache, table.cuda(), ints(lens).cuda())
        jobs.append((args, api.cache_attention(*args)[0], api.cache_read(*args[1:], 50), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        for args, _, _, stream in jobs:
            got.append((api.cache_attention(*args, stream=stream)[0], api.cache_read(*args[1:], 50, stream=stream)))
    torch.cuda.synchronize()
    api.poll_status()
    for n, (out, (k, v)) in enumerate(got):
        _, want, (wk, wv), _ = jobs[n % 2]
        assert torch.equal(out, want) and torch.equal(k, wk) and torch.equal(v, wv)


@pytest.mark.gpu
def test_a_growing_sequence_keeps_its_tokens():
    """Tokens written one call at a time, across tile and page ends, against one call for all."""
    rng = np.random.default_rng(34)
    B, H, D, page, n = 2, 2, 96, 16, 37
    table = ints([[3, 0, 5], [1, 4, 2]]).cuda()
    k, v = (draw_rows(rng, (B, H, n, D), "f16").cuda() for _ in range(2))
    once, grown = dirty_cache(6, H, page, D, "f16"), dirty_cache(6, H, page, D, "f16")
    api.cache_write(once, k, v, table, ints([n, n]).cuda())
    at = 0
    for rows in (1, 1, 14, 2, 15, 3, 1):
        api.cache_write(grown, k[:, :, at:at + rows], v[:, :, at:at + rows], table, ints([at + rows] * B).cuda())
        at += rows
    api.poll_status()
    assert at == n and torch.equal(once.view(torch.uint8), grown.view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("D,G", [(32, 4), (128, 1), (128, 8), (64, 16)])
def test_a_nan_key_reaches_out_and_lse(D, G):
    """The newest token's key holds a NaN: the rows that see it are NaN in out and lse, alone in
    its unit, as the only token, or beside finite ones of the same unit; the others are not."""
    rng = np.random.default_rng(35)
    unit = 64 if D <= 64 else 32
    lens, H, L = [1, unit + 1, 3 * unit + 5, 700, 0], 2, 2
    cache, table, ks, vs, low = fill(rng, lens, H, D, 32, "bf16")
    q = draw_rows(rng, (len(lens), G * H, L, D), "bf16").cuda()
    args = (q, cache, table.cuda(), ints(lens).cuda())
    bad = torch.full((len(lens), H, 1, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    api.cache_write(cache, bad, bad, *args[2:])
    out, lse = api.cache_attention(*args, need_lse=True)
    api.poll_status()
    for b, n in enumerate(lens):
        assert bool(out[b, :, 1].isnan().all()) == (n > 0) and bool(lse[b, :, 1].isnan().all()) == (n > 0), n
    before = [[x[:, :max(0, n - 1)] for x, n in zip(xs, lens)] for xs in (ks, vs, low)]
    check(out[:, :, :1], lse[:, :, :1], q[:, :, :1], *before, 1 / math.sqrt(D), True, None, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("B,H,G", [(1, 1, 1), (40, 8, 8)])
def test_constant_values_under_rising_scores(B, H, G, dtype):
    """Values whose groups are constant (scale 0), and scores that rise by 8 in base 2, as far as
    a row's reference may lag, from one unit of a warp to its next: every output is the constant."""
    D, page, rise = 32, 64, 256 if G <= 4 else 512                     # 4 or 8 warps of units of 64
    n = 2 * rise
    k = torch.zeros(B, H, n, D, dtype=TYPES[dtype])
    k[..., 1] = 15.0                                                   # scale 1, zero 0: exact codes
    k[:, :, rise:, 0] = 8.0
    v = torch.full_like(k, 1.5)
    table = torch.arange(B * n // page, dtype=torch.int32).view(B, n // page).cuda()
    lens = ints([n] * B).cuda()
    cache = dirty_cache(B * n // page, H, page, D, dtype)
    api.cache_write(cache, k.cuda(), v.cuda(), table, lens)
    q = torch.zeros(B, H * G, 1, D, dtype=TYPES[dtype], device="cuda")
    q[..., 0] = 1.0
    out, lse = api.cache_attention(q, cache, table, lens, scale=math.log(2), need_lse=True)
    api.poll_status()
    want = math.log(rise * (1 + 2.0**8))
    assert bool((out == 1.5).all())                                    # 2^-16·1.5 is less than half a step
    assert np.abs(as_f64(lse) - want).max() <= 2.0**-16 * want


@pytest.mark.gpu
def test_a_strided_workspace_is_refused():
    cache = api.cache_empty(300, 1, 16, 64)
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    table, lens = torch.arange(300, dtype=torch.int32, device="cuda").view(1, 300), ints([0]).cuda()
    for ws in (torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 16), torch.empty(1 << 18, device="cuda")[::4]):
        with pytest.raises(ValueError):
            api.cache_attention(q, cache, table, lens, workspace=ws)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,G,L", [(32, 4, 1), (96, 1, 3), (128, 4, 1), (256, 16, 1)])
def test_scores_keep_fp32_precision(D, G, L, dtype):
    """lse of sequences of one token is the score itself.  D/32 groups, each a sum of 32 products
    and a z term about twice as large as what is left of them: fp32 sums are off by some 2^-24 of
    those terms' root sum, 2^-24·3·sqrt(D) against a score of sqrt(D)·|q||k|, and bf16 may be 4 times
    that (its codes' lower nibbles are summed with up to 4 bits fewer): rms relative errors of
    2^-22 and 2^-20."""
    rng = np.random.default_rng(36)
    B, H = 16, 8
    cache, table, ks, vs, low = fill(rng, [1] * B, H, D, 16, dtype)
    q = draw_rows(rng, (B, G * H, L, D), dtype)
    _, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints([1] * B).cuda(), need_lse=True, is_causal=False)
    _, want = ref.cached_attention(as_f64(q), ks, vs, 1 / math.sqrt(D), False, None)
    assert np.linalg.norm(as_f64(lse) - want) <= (2.0**-22 if dtype == "f16" else 2.0**-20) * np.linalg.norm(want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,G,L", [(32, 2, 1), (64, 4, 1), (96, 1, 2), (128, 4, 1), (256, 1, 1), (64, 8, 1), (128, 5, 1), (256, 2, 4), (96, 4, 4), (128, 8, 2)])
def test_lengths_that_end_anywhere(D, G, L, dtype):
    """Every length from 0 to two units and a little: ends inside tiles, halves and units of every
    form, where the lanes of a warp differ in what they see."""
    rng = np.random.default_rng(43)
    lens = list(range(0, 70 if D > 64 else 132, 1 if D > 64 else 3))
    cache, table, ks, vs, low = fill(rng, lens, 1, D, 16, dtype)
    q = draw_rows(rng, (len(lens), G, L, D), dtype)
    out, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints(lens).cuda(), need_lse=True)
    api.poll_status()
    check(out, lse, q, ks, vs, low, 1 / math.sqrt(D), True, None, dtype)


def sizes(q, ks, vs, low, scale, causal, sink):
    """sum_j w_j·(|z| + s·c) of every output element: what its fp32 sums are made of."""
    return ref.cached_attention(as_f64(q), ks, [np.abs(v - x) + x for v, x in zip(vs, low)], scale, causal, sink)[0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,G,L", [(128, 4, 1), (32, 2, 2), (128, 8, 1), (96, 5, 1), (64, 4, 4), (128, 4, 8), (256, 1, 1), (256, 16, 1)])
def test_outputs_are_rounded_once(D, G, L, dtype):
    """P·s is as good as fp32: an output differs from the rounded exact one only where that lies
    close to the middle of two numbers.  With |S| of a few units an output is off by less than
    off = 2^-19·sum_j w_j·(|z| + s·c) before it is rounded (2^-20 the sums of the MMA, where lower
    nibbles keep fewer low bits, 2^-21 P·s, 2^-22 twice the scores and what follows from them), so
    that the odds of an element are 2·off / step; their sum over all elements, and 4 standard
    deviations, bounds how many differ.  (P·s rounded to 2^-11 changes one bf16 output in six.)"""
    rng = np.random.default_rng(37)
    lens, H = [100, 61, 33, 128], 2
    cache, table, ks, vs, low = fill(rng, lens, H, D, 16, dtype)
    q = draw_rows(rng, (len(lens), G * H, L, D), dtype, 0.5)
    out, _ = api.cache_attention(q.cuda(), cache, table.cuda(), ints(lens).cuda())
    api.poll_status()
    o, _ = ref.cached_attention(as_f64(q), ks, vs, 1 / math.sqrt(D), True, None)
    off = 2.0**-19 * sizes(q, ks, vs, low, 1 / math.sqrt(D), True, None)
    step = torch.finfo(TYPES[dtype]).eps * np.exp2(np.floor(np.log2(np.abs(o))))
    odds = np.minimum(1, 2 * off / step).sum()
    differ = (as_f64(out) != ref.rounded(o, TYPES[dtype])).sum()
    assert differ <= odds + 4 * math.sqrt(odds) + 1, f"{differ} of {o.size} differ, {odds:.1f} expected at most"


@pytest.mark.gpu
@pytest.mark.parametrize("D,G,L", [(32, 4, 1), (96, 1, 3), (128, 4, 1), (128, 8, 1), (256, 16, 1)])
def test_bf16_scores_keep_fp32_precision(D, G, L):
    """The same, and the same bound as fp16's, for bf16: the sums over its codes' lower nibbles lose
    nothing either."""
    rng = np.random.default_rng(38)
    B, H = 16, 8
    cache, table, ks, vs, low = fill(rng, [1] * B, H, D, 16, "bf16")
    q = draw_rows(rng, (B, G * H, L, D), "bf16")
    _, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints([1] * B).cuda(), need_lse=True, is_causal=False)
    api.poll_status()
    _, want = ref.cached_attention(as_f64(q), ks, vs, 1 / math.sqrt(D), False, None)
    assert np.linalg.norm(as_f64(lse) - want) <= 2.0**-22 * np.linalg.norm(want)


@pytest.mark.gpu
@pytest.mark.parametrize("D,G,L", [(128, 4, 1), (64, 8, 1), (128, 2, 8)])
def test_a_nan_value_without_weight_is_nan_wherever_it_lies(D, G, L):
    """A visible key whose probability is 0 (a score of -1000) and whose values of one group are
    NaN: 0·NaN is NaN, in a whole unit as in one that the sequence's or a query's end cuts; the
    queries before it do not see it."""
    rng = np.random.default_rng(39)
    H, page = 2, 32
    lens = [200, 200, 200, 33]
    bad = [10, 150, 199, 32]                                           # its position: inside, and last
    table, pages = make_table(rng, lens, page)
    cache = dirty_cache(pages, H, page, D, "bf16")
    k, v = (draw_rows(rng, (len(lens), H, 200, D), "bf16") for _ in range(2))
    k[..., 0] = 0
    for b, n in enumerate(lens):
        k[b, :, 200 - n + bad[b], 0] = -1000 * math.sqrt(D)
        v[b, :, 200 - n + bad[b], 37] = float("nan")
    q = draw_rows(rng, (len(lens), G * H, L, D), "bf16")
    q[..., 0] = 1.0
    api.cache_write(cache, k.cuda(), v.cuda(), table.cuda(), ints(lens).cuda())
    out, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints(lens).cuda(), need_lse=True)
    api.poll_status()
    assert torch.isfinite(lse).all() and torch.isfinite(out[..., :32]).all() and torch.isfinite(out[..., 64:]).all()
    for b, n in enumerate(lens):
        for i in range(L):
            got = out[b, :, i, 32:64].isnan()
            assert bool(got.all()) if n - L + i >= bad[b] else not bool(got.any()), (b, i)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [None, 1.0, -0.25, 1e30, 1e-30])
@pytest.mark.parametrize("D,G,L", [(32, 4, 1), (128, 8, 1), (64, 4, 4), (256, 2, 1)])
def test_queries_up_to_the_largest(D, G, L, scale):
    """Rows of 2^90 to bf16's largest numbers, and tiny ones, whose scores are ordinary because the
    keys are small, and keys of zero, whose scores are 0 whatever the query and the scale."""
    rng = np.random.default_rng(40)
    H, n = 1, 70
    used = 1 / math.sqrt(D) if scale is None else scale
    for power in (127, 126, 120, 90, -100):
        key = -power - math.log2(abs(used)) + 1.0 - math.log2(D) / 2   # |S| of a few units
        for zero in (False, True):
            if not zero and abs(key) > 118:
                continue
            table, pages = make_table(rng, [n], 16)
            cache = dirty_cache(pages, H, 16, D, "bf16")
            v = draw_rows(rng, (1, H, n, D), "bf16")
            k = torch.zeros_like(v) if zero else (draw_rows(rng, (1, H, n, D), "bf16").double() * 2.0**key).to(v.dtype)
            # Uniform in (-1, 1), so that no element passes the type's largest number; the first row is plain.
            q = torch.from_numpy(rng.uniform(-1, 1, (1, G * H, L, D))) * 2.0**power
            q[:, 0] *= 2.0**-power * 2.0**min(power, 60)
            q = q.to(v.dtype)
            api.cache_write(cache, k.cuda(), v.cuda(), table.cuda(), ints([n]).cuda())
            out, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints([n]).cuda(), scale=scale, need_lse=True)
            api.poll_status()
            code, s, z = ref.quantise(as_f64(v)[0], torch.bfloat16)
            ks, vs, low = [held(as_f64(k)[0], "bf16")], [ref.values(code, s, z)], [ref.values(code, s, np.zeros_like(z))]
            check(out, lse, q, ks, vs, low, float(np.float32(used)), True, None, "bf16")


def check_groups(out, q, ks, vs, low, scale, causal, dtype, what):
    """Every element against its own group: eps(T)/2·|o| for its rounding (2^-25 where fp16 has no
    smaller step) and 2^-15·sum_j w_j·(|z| + s·c), the scores' error (|S| of 20 to 100, 2^-22 and
    less of them, twice with the sum) on what it is made of, and on nothing larger."""
    o, _ = ref.cached_attention(as_f64(q), ks, vs, scale, causal, None)
    tol = torch.finfo(TYPES[dtype]).eps / 2 * np.abs(o) + 2.0**-15 * sizes(q, ks, vs, low, scale, causal, None) + (2.0**-25 if dtype == "f16" else 0)
    worst = (np.abs(as_f64(out) - o) / np.maximum(tol, 1e-300)).max()
    assert np.isfinite(as_f64(out)).all() and worst <= 1, f"{what}: {worst:.2f} of the tolerance"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,large,plain", [("bf16", 1e30, 1.0), ("bf16", 1.0, 1e-25), ("f16", 5e3, 2e-3)])
@pytest.mark.parametrize("D,G,L", [(128, 4, 1), (128, 8, 1), (64, 2, 4), (32, 4, 8), (256, 4, 1), (96, 3, 3)])
def test_values_that_a_row_does_not_weigh(D, G, L, dtype, large, plain):
    """A key with large values leaves the rows alone that do not see it (it is the newest, and they
    are earlier) and those for which its weight is negligible (a score of -100, or -60 in fp16,
    below the others), wherever it lies; and in one group of 32 values only, or in all."""
    rng = np.random.default_rng(41)
    H, page, n, scale = 1, 64, 1400, 1 / math.sqrt(D)
    below = 100 if dtype == "bf16" else 60
    for at, group in ((n - 1, False), (3, False), (40, True), (700, False), (n - 1, True), (n - 5, False)):
        table, pages = make_table(rng, [n], page)
        cache = dirty_cache(pages, H, page, D, dtype)
        k, v = (draw_rows(rng, (1, H, n, D), dtype) for _ in range(2))
        v = (v.double() * plain).to(v.dtype)
        k[..., 0] = 0
        k[:, :, at, 0] = -below / scale / 8
        where = slice(D - 32, D) if group else slice(None)
        v[:, :, at, where] = (draw_rows(rng, v[:, :, at, where].shape, dtype).double() * large).to(v.dtype)
        q = draw_rows(rng, (1, G * H, L, D), dtype)
        q[..., 0] = 8
        api.cache_write(cache, k.cuda(), v.cuda(), table.cuda(), ints([n]).cuda())
        out, _ = api.cache_attention(q.cuda(), cache, table.cuda(), ints([n]).cuda())
        api.poll_status()
        code, s, z = ref.quantise(as_f64(v)[0], TYPES[dtype])
        ks, vs, low = [held(as_f64(k)[0], dtype)], [ref.values(code, s, z)], [ref.values(code, s, np.zeros_like(z))]
        check_groups(out, q, ks, vs, low, scale, True, dtype, f"key {at}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,large,small", [("bf16", 1.0, 2.0**-26), ("bf16", 2.0**100, 2.0**-100), ("f16", 2.0**13, 2.0**-11)])
@pytest.mark.parametrize("D,G,L", [(128, 4, 1), (128, 8, 1), (64, 4, 4), (256, 2, 1)])
def test_groups_far_apart_in_size(D, G, L, dtype, large, small):
    """Groups of small values beside groups of large ones keep their own precision, also where
    scores and scales rise along the sequence."""
    rng = np.random.default_rng(42)
    H, page, n, scale = 2, 32, 500, 1 / math.sqrt(D)
    for rising in (False, True):
        table, pages = make_table(rng, [n], page)
        cache = dirty_cache(pages, H, page, D, dtype)
        k, v = (draw_rows(rng, (1, H, n, D), dtype) for _ in range(2))
        v = v.double() * large
        v[..., :32] *= small / large
        if rising:
            v *= torch.exp2(-torch.arange(n - 1, -1, -1).double() // 100 * 2).view(1, 1, n, 1)
            k[..., 0] = torch.linspace(-20, 20, n).to(k.dtype)
        v = v.to(k.dtype)
        q = draw_rows(rng, (1, G * H, L, D), dtype)
        q[..., 0] = 1 / scale
        api.cache_write(cache, k.cuda(), v.cuda(), table.cuda(), ints([n]).cuda())
        out, _ = api.cache_attention(q.cuda(), cache, table.cuda(), ints([n]).cuda())
        api.poll_status()
        code, s, z = ref.quantise(as_f64(v)[0], TYPES[dtype])
        ks, vs, low = [held(as_f64(k)[0], dtype)], [ref.values(code, s, z)], [ref.values(code, s, np.zeros_like(z))]
        check_groups(out, q, ks, vs, low, scale, True, dtype, f"rising {rising}")


@pytest.mark.parametrize("B,Hq,Hkv,L,D", [(1, 32, 8, 4096, 128), (1, 32, 8, 512, 128), (1, 4, 1, 1, 128), (4096, 32, 8, 1, 64), (64, 64, 8, 16, 256), (2, 16, 1, 1024, 32)])
@pytest.mark.parametrize("tokens", [2048, 131072, 1 << 30])
def test_the_workspace_stays_small(B, Hq, Hkv, L, D, tokens):
    """Partial results of all rows take 64 MiB at most, however wide the table is."""
    build.build()
    page = 16384 if tokens > 131072 else 128
    c = _lib.Cache(*dict(GOOD, num_pages=4, page_size=page, Hkv=Hkv, D=D, pages_stride=tokens // page, pages_per_seq=tokens // page).values())
    assert _lib.sdpa_cache_attn_workspace_size(c, B, Hq, L, 0) <= 64 << 20


@pytest.mark.gpu
def test_many_rows_and_a_wide_table():
    """Rows enough that the workspace's bound sets the chunks, on a table far wider than the
    sequences: one of three chunks, an empty one, and one of a few tokens."""
    rng = np.random.default_rng(44)
    lens, Hq, L, D, page = [20000, 0, 40], 16, 700, 32, 1024
    cache, table, ks, vs, low = fill(rng, lens, 1, D, page, "bf16", width=128)
    q = draw_rows(rng, (3, Hq, L, D), "bf16")
    c = api._cache(cache, table.cuda(), ints(lens).cuda(), 3)
    assert 32 << 20 < _lib.sdpa_cache_attn_workspace_size(c, 3, Hq, L, 0) <= 64 << 20
    out, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints(lens).cuda(), need_lse=True)
    api.poll_status()
    rows = [0, 1, 350, 660, 661, 698, 699]                              # 660: the first that sees one of 40
    for i in rows:                                                      # a row is the last one of a sequence cut behind it
        seen = [[x[:, :max(0, n - L + i + 1)] for x, n in zip(xs, lens)] for xs in (ks, vs, low)]
        check(out[:, :, i:i + 1], lse[:, :, i:i + 1], q[:, :, i:i + 1], *seen, 1 / math.sqrt(D), True, None, "bf16")


@pytest.mark.gpu
def test_a_bound_past_32_bits_is_no_bound():
    """max_len beyond every length, as large as a Python integer may be, changes nothing."""
    rng = np.random.default_rng(46)
    cache, table, *_ = fill(rng, [90, 17], 2, 64, 16, "bf16")
    q = draw_rows(rng, (2, 4, 1, 64), "bf16").cuda()
    args = (q, cache, table.cuda(), ints([90, 17]).cuda())
    want, _ = api.cache_attention(*args)
    for most in (2**31 - 1, 2**31, 2**32 + 1, 2**63, 5 - 2**32):         # 0 and less: the table's end
        assert torch.equal(api.cache_attention(*args, max_len=most)[0], want)
    api.poll_status()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("G,L", [(4, 1), (8, 1), (4, 4)])
@pytest.mark.parametrize("D", [32, 64, 96, 256])
@pytest.mark.parametrize("lens", [[3000, 700, 0, 1025], [20000, 5]])
def test_sequences_of_several_chunks(lens, D, G, L, dtype):
    """Joins of a few chunks by four warps and of many by sixteen, with the head dims whose rows do
    and do not divide a block's threads, in every form."""
    rng = np.random.default_rng(45)
    cache, table, ks, vs, low = fill(rng, lens, 1, D, 64, dtype)
    q = draw_rows(rng, (len(lens), G, L, D), dtype)
    sink = torch.from_numpy(rng.standard_normal(G).astype(np.float32)).cuda()
    c = api._cache(cache, table.cuda(), ints(lens).cuda(), len(lens))
    splits = _lib.sdpa_cache_attn_workspace_size(c, len(lens), G, L, 0) // (len(lens) * G * L * (D + 2) * 4)
    assert splits > 16 if max(lens) > 3000 else 1 < splits <= 16
    out, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints(lens).cuda(), need_lse=True, sinks=sink)
    api.poll_status()
    check(out, lse, q, ks, vs, low, 1 / math.sqrt(D), True, sink.cpu().numpy(), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("D,G,L", [(64, 4, 1), (128, 8, 1), (64, 8, 2)])
def test_scores_that_fp32_holds_coarsely(D, G, L):
    """Scores of 2^20 to 2^28, where one step of fp32 (in base 2) is up to 32: the largest key alone has weight,
    whatever a row's reference is rounded to."""
    rng = np.random.default_rng(47)
    n, page = 200, 16
    table, pages = make_table(rng, [n], page)
    cache = dirty_cache(pages, 1, page, D, "bf16")
    v = draw_rows(rng, (1, 1, n, D), "bf16")
    size = torch.from_numpy(rng.uniform(0.25, 0.5, (1, 1, n, 1))).to(v.dtype)
    size[0, 0, [3, 77, 190]] = 1.0                                     # ties, exactly
    api.cache_write(cache, size.expand(1, 1, n, D).contiguous().cuda(), v.cuda(), table.cuda(), ints([n]).cuda())
    code, s, z = ref.quantise(as_f64(v)[0], torch.bfloat16)
    ks, vs, low = [as_f64(size.expand(1, 1, n, D))[0]], [ref.values(code, s, z)], [ref.values(code, s, np.zeros_like(z))]
    for power in (20, 24, 28):
        q = torch.full((1, G * 1, L, D), 1.0) * 2.0**power * torch.from_numpy(rng.uniform(0.5, 1, (1, G, L, 1)))
        q = q.to(v.dtype)
        out, lse = api.cache_attention(q.cuda(), cache, table.cuda(), ints([n]).cuda(), scale=1 / D, need_lse=True, is_causal=False)
        api.poll_status()
        check(out, lse, q, ks, vs, low, 1 / D, False, None, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("G,L", [(4, 1), (8, 1), (4, 4)])
def test_sums_over_long_sequences(G, L):
    """100000 tokens, whose outputs are some 300 times smaller than one value.  A chain of 64 MMAs,
    each of which may cut off 2^-23 of its sum, is off by 2^-17 of that sum at most, and the sums are
    no larger than the outputs' random part r = sqrt(sum_j w_j²·(s·(c - 8))²), a few times, and the
    output itself: off = 2^-17·(3·r + |o|).  Odds as in ``test_outputs_are_rounded_once``.  (Codes
    of 0 to 15 add up to 500 times an output, and change one in seven.)"""
    rng = np.random.default_rng(48)
    n, D = 100000, 32
    table, pages = make_table(rng, [n], 1024)
    cache = dirty_cache(pages, 1, 1024, D, "bf16")
    k, v = (draw_rows(rng, (1, 1, n, D), "bf16") for _ in range(2))
    api.cache_write(cache, k.cuda(), v.cuda(), table.cuda(), ints([n]).cuda())
    q = draw_rows(rng, (1, G, L, D), "bf16")
    out, _ = api.cache_attention(q.cuda(), cache, table.cuda(), ints([n]).cuda(), is_causal=False)
    api.poll_status()
    code, s, _ = ref.quantise(as_f64(v)[0, 0], torch.bfloat16)
    weight = as_f64(q)[0].reshape(-1, D) @ held(as_f64(k)[0, 0], "bf16").T / math.sqrt(D)
    weight = np.exp(weight - weight.max(1, keepdims=True))
    weight /= weight.sum(1, keepdims=True)
    o = weight @ held(as_f64(v)[0, 0], "bf16")
    r = np.sqrt(weight**2 @ (s * (code - 8.0))**2)
    step = torch.finfo(torch.bfloat16).eps * np.exp2(np.floor(np.log2(np.abs(o))))
    odds = np.minimum(1, 2.0**-16 * (3 * r + np.abs(o)) / step).sum()
    differ = (as_f64(out)[0].reshape(-1, D) != ref.rounded(o, torch.bfloat16)).sum()
    assert differ <= odds + 4 * math.sqrt(odds) + 1, f"{differ} of {o.size} differ, {odds:.1f} expected at most"
