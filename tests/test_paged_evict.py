"""Attention weights of a 16-bit paged cache's tokens and eviction by them, against the fp64 oracle,
and the cache's operators as they are used together.

Tolerance of a weight: (2·ds + 2^-20 + (rows + 8)·2^-24)·gain + 2^-23·(old + gain), where a
probability is off by ds = (D + 8)·2^-24·S + 2^-23·|lse| relative to itself (its score, D products
summed in fp32 of size S = sum |q·k|·scale at most, and its lse, multiplied by log2(e) as one number
at worst) and the exponential by 2^-21."""
import math

import numpy as np
import pytest
import torch

from cache_util import TYPES, draw_rows, ints, make_table
from oracle import paged as ref
from paged_util import NAN, check, dirty, fill, on_device
from scaled_dot_product_flash_gb300 import _lib, api
from scaled_dot_product_flash_gb300.inputs import as_f64
from test_paged_attention import BAD_CACHES, CASES, COUNTS, GOOD, LSE, OUT, Q, cache_of

INVALID, UNSUPPORTED, WORKSPACE, INDEX = 1, 2, 5, 6
WEIGHTS, KEPT, NEW_LENS = OUT, LSE, COUNTS


def check_weights(got, q, ks, vs, lse, old, scale, causal, counts=None):
    got, old, lse = as_f64(got), as_f64(old), as_f64(lse)
    want, gain = ref.weights(as_f64(q), ks, lse, old, scale, causal, counts)
    S = ref.attention(as_f64(q), ks, vs, scale, causal, counts)[3].max()
    top = np.abs(lse[np.isfinite(lse)]).max(initial=0)
    rows = q.shape[1] // ks[0].shape[0] * q.shape[2]
    ds = (q.shape[3] + 8) * 2.0**-24 * S + 2.0**-23 * top
    tol = (2 * ds + 2.0**-20 + (rows + 8) * 2.0**-24) * gain + 2.0**-23 * np.abs(want) + 1e-30
    worst = (np.abs(got - want) / tol).max()
    assert worst <= 1, f"weights are {worst:.2f} of their tolerance"


# ---- without a GPU


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(q=0), INVALID), (dict(q=Q + 8), INVALID), (dict(lse=0), INVALID), (dict(lse=LSE + 2), INVALID), (dict(weights=0), INVALID),
    (dict(weights=WEIGHTS + 1), INVALID), (dict(counts=COUNTS + 1), INVALID), (dict(lay=None), INVALID), (dict(lay=(256, 64, 60)), INVALID),
    (dict(ws=None), INVALID), (dict(ws=(0, 100)), INVALID), (dict(ws=(199, 100)), INVALID), (dict(ws=(200, 99)), INVALID), (dict(ws=(-200, 100)), INVALID),
    (dict(slots=0), INVALID), (dict(scale=NAN), INVALID), (dict(causal=1), UNSUPPORTED), (dict(causal=4), INVALID), (dict(Hq=3), INVALID),
    (dict(Lq=0), INVALID), (dict(weights=Q), INVALID), (dict(weights=LSE), INVALID), (dict(weights=GOOD["data"] + 64), INVALID),
    (dict(weights=GOOD["lens"]), INVALID), (dict(weights=GOOD["pages"]), INVALID), (dict(weights=COUNTS), INVALID)])
def test_weights_refused(kw, code):
    a = dict(GOOD, q=Q, lse=LSE, weights=WEIGHTS, ws=(200, 100), slots=100, lay=(256, 64, 64), counts=COUNTS, B=2, Hq=4, Lq=1, scale=0.125, causal=2)
    a.update(kw)
    lay = None if a["lay"] is None else _lib.Int64x3(*a["lay"])
    ws = None if a["ws"] is None else api._pack2(*a["ws"])
    assert _lib.sdpa_paged_weights(cache_of(a), a["q"], a["lse"], a["weights"], ws, a["slots"], lay, a["counts"], a["B"], a["Hq"], a["Lq"], a["scale"],
                                   a["causal"], 0, None) == code


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(w=0), INVALID), (dict(nw=0), INVALID), (dict(w=WEIGHTS + 2), INVALID), (dict(nw=Q + 1), INVALID), (dict(new_lens=0), INVALID),
    (dict(new_lens=NEW_LENS + 1), INVALID), (dict(kept=0), INVALID), (dict(kept=KEPT + 3), INVALID), (dict(ws=None), INVALID),
    (dict(ws=(0, 100, 200, 100)), INVALID), (dict(ws=(200, 100, 200, 50)), INVALID), (dict(slots=0), INVALID), (dict(budget=0), INVALID),
    (dict(budget=-1), INVALID), (dict(recent=-1), INVALID), (dict(recent=51), INVALID), (dict(nw=WEIGHTS, ws=(200, 100, 400, 100)), INVALID),
    (dict(nw=WEIGHTS + 4), INVALID), (dict(new_lens=GOOD["lens"] + 4), INVALID), (dict(kept=WEIGHTS), INVALID), (dict(kept=GOOD["data"]), INVALID),
    (dict(nw=GOOD["data"]), INVALID), (dict(w=GOOD["data"]), INVALID), (dict(kept=GOOD["lens"]), INVALID), (dict(kept=GOOD["pages"]), INVALID),
    (dict(new_lens=GOOD["pages"]), INVALID), (dict(new_lens=KEPT), INVALID), (dict(nw=KEPT), INVALID), (dict(Hkv=40000), UNSUPPORTED)])
def test_evict_refused(kw, code):
    a = dict(GOOD, w=WEIGHTS, nw=Q, ws=(200, 100, 200, 100), slots=100, new_lens=NEW_LENS, kept=KEPT, B=2, budget=50, recent=10)
    a.update(kw)
    if a["Hkv"] == 40000:
        a["ws"] = (4000000, 100, 4000000, 100)
    ws = None if a["ws"] is None else api._pack4(*a["ws"])
    assert _lib.sdpa_paged_evict(cache_of(a), a["w"], a["nw"], ws, a["slots"], a["new_lens"], a["kept"], a["B"], a["budget"], a["recent"], None) == code


# ---- weights, on the GPU


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,Hq,Hkv,L,D,page,lens,counts", CASES)
def test_weights(dtype, Hq, Hkv, L, D, page, lens, counts, causal):
    rng = np.random.default_rng(1000 * L + D + len(lens))
    cache, table, ks, vs = fill(rng, lens, Hkv, D, page, dtype)
    q = draw_rows(rng, (len(lens), Hq, L, D), dtype, 1.5)
    at, dev_counts = on_device(table, lens, counts)
    how = dict(is_causal="bottom_right" if causal else False, counts=dev_counts)
    sinks = torch.from_numpy(rng.standard_normal(Hq).astype(np.float32)).cuda() if L % 2 else None
    _, lse = api.paged_attention(q.cuda(), cache, *at, need_lse=True, sinks=sinks, **how)
    wide = torch.from_numpy(rng.random((Hkv, len(lens), max(lens) + 9)).astype(np.float32)).cuda()
    weights = wide[..., 2:-3].transpose(0, 1)                                    # heads outermost, unaligned rows
    old, before = weights.clone(), wide.clone()
    assert api.paged_weights(q.cuda(), cache, *at, lse, weights, **how) is weights
    api.poll_status()
    check_weights(weights, q, ks, vs, lse, old, 1 / math.sqrt(D), causal, counts)
    for b, n in enumerate(lens):                                                 # slots behind a sequence, and beside the rows
        assert torch.equal(weights[b, :, n:], old[b, :, n:])
    assert torch.equal(wide[..., :2], before[..., :2]) and torch.equal(wide[..., -3:], before[..., -3:])


@pytest.mark.gpu
@pytest.mark.parametrize("L", [1, 7, 90])
def test_fresh_slots_hold_anything(L):
    """The slots of the call's own tokens are NaN before it; two calls give the same bits."""
    rng = np.random.default_rng(11)
    lens, counts = [200, L, 95], [L, L, max(1, L // 2)]
    cache, table, ks, vs = fill(rng, lens, 2, 64, 16, "bf16")
    q = draw_rows(rng, (3, 8, L, 64), "bf16")
    at, dev_counts = on_device(table, lens, counts)
    _, lse = api.paged_attention(q.cuda(), cache, *at, need_lse=True, counts=dev_counts)
    old = torch.rand(3, 2, 210, device="cuda")
    clean = old.clone()
    for b, n in enumerate(lens):
        old[b, :, n - counts[b]:] = NAN
        clean[b, :, n - counts[b]:] = 0
    got = [api.paged_weights(q.cuda(), cache, *at, lse, old.clone(), counts=dev_counts) for _ in range(2)]
    api.poll_status()
    live = torch.stack([torch.arange(210, device="cuda") < n for n in lens]).unsqueeze(1)
    assert torch.equal(got[0].nan_to_num(-1.0), got[1].nan_to_num(-1.0))
    check_weights(torch.where(live, got[0], clean), q, ks, vs, lse, clean, 1 / 8, True, counts)
    assert got[0][~live.expand_as(old)].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("L", [3, 70])
def test_rows_without_weight_and_hidden_nan(L):
    """Rows whose lse is -inf add nothing, whatever their queries; a NaN key is NaN for itself alone."""
    rng = np.random.default_rng(12)
    n = L + 50
    cache, table, ks, vs = fill(rng, [n], 1, 64, 16, "f16")
    q = draw_rows(rng, (1, 4, L, 64), "f16")
    at, _ = on_device(table, [n])
    _, lse = api.paged_attention(q.cuda(), cache, *at, need_lse=True)
    lse[:, 1] = -float("inf")
    bad = q.clone()
    bad[:, 1] = NAN
    cache[table[0, 1], 0, 0, 3] = NAN                                            # token 19
    got = api.paged_weights(bad.cuda(), cache, *at, lse, torch.zeros(1, 1, n, device="cuda"))
    api.poll_status()
    assert got[0, 0, 19].isnan()
    want = ref.weights(as_f64(q), ks, as_f64(lse), np.zeros((1, 1, n)), 1 / 8, True)[0]
    got[0, 0, 19] = want[0, 0, 19]
    assert np.abs(as_f64(got) - want).max() <= 2.0**-14 * want.max()


@pytest.mark.gpu
def test_weights_beyond_the_slots():
    rng = np.random.default_rng(13)
    cache, table, ks, vs = fill(rng, [50], 1, 32, 16, "f16")
    q = draw_rows(rng, (1, 2, 1, 32), "f16").cuda()
    at, _ = on_device(table, [50])
    _, lse = api.paged_attention(q, cache, *at, need_lse=True)
    wide = torch.zeros(1, 1, 60, device="cuda")
    api.paged_weights(q, cache, *at, lse, wide[..., :40])                        # the sequence is longer than its slots
    with pytest.raises(_lib.SdpaError) as e:
        api.poll_status()
    assert e.value.status == INDEX and not wide[..., 40:].any()


# ---- eviction, on the GPU


def evicted(cache, table, lens, weights, budget, recent):
    """What is expected: (cache, lens, weights, kept) on the CPU."""
    cache, page = cache.cpu().clone(), cache.shape[3]
    B, H, slots = weights.shape
    new = torch.zeros(weights.shape)
    kept = torch.full((B, H, budget), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        at = [(int(table[b, j // page]), j % page) for j in range(n)]
        for h in range(H):
            stay = ref.kept(weights[b, h].cpu().numpy(), n, budget, recent)
            kept[b, h, :len(stay)] = torch.tensor(stay, dtype=torch.int32)
            new[b, h, :len(stay)] = weights[b, h].cpu()[stay]
            rows = [cache[at[j][0], :, h, at[j][1]].clone() for j in stay]
            for r, x in enumerate(rows):
                cache[at[r][0], :, h, at[r][1]] = x
    return cache, ints([min(n, budget) for n in lens]), new, kept


def same(got, want):
    for x, y in zip(got, want):
        x = x.cpu()
        if x.dtype in (torch.float16, torch.bfloat16):
            x, y = x.view(torch.int16), y.view(torch.int16)
        if x.dtype is torch.float32:
            x, y = x.view(torch.int32), y.contiguous().view(torch.int32)
        assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype,H,D,page,lens,budget,recent", [
    ("bf16", 1, 32, 16, [1], 1, 0),
    ("f16", 2, 64, 16, [0, 1, 16, 17, 40], 16, 4),
    ("bf16", 3, 128, 48, [300, 10, 150], 100, 100),                # nothing but recent tokens
    ("bf16", 2, 96, 32, [333, 200], 199, 0),
    ("f16", 1, 256, 64, [129, 128, 64], 128, 17),
    ("bf16", 8, 128, 16, [70] * 5, 1, 1),
    ("f16", 1, 64, 80, [5000, 4097], 2500, 300),
])
def test_evict(dtype, H, D, page, lens, budget, recent, in_place):
    rng = np.random.default_rng(D + budget)
    cache, table, _, _ = fill(rng, lens, H, D, page, dtype)
    slots = max(lens) + 3
    w = np.exp(rng.standard_normal((len(lens), H, slots))).astype(np.float32)
    w[rng.random(w.shape) < 0.3] = 0.5                                           # ties
    at, _ = on_device(table, lens)
    weights = torch.from_numpy(w).cuda()
    want = evicted(cache, table, lens, weights, budget, recent)
    if in_place:
        out = api.paged_evict(cache, *at, weights, budget, recent, new_lens=at[1], new_weights=weights)
        assert out[0] is at[1] and out[1] is weights
    else:
        before = weights.clone()
        out = api.paged_evict(cache, *at, weights, budget, recent)
        assert torch.equal(weights, before) and at[1].tolist() == lens
    api.poll_status()
    same((cache, *out), want)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,budget,recent", [([700, 300], 200, 40), ([9000, 100], 3000, 2900)])
def test_evict_rows_of_a_larger_tensor(lens, budget, recent):
    """Weights with the heads outermost and rows off the 16-byte grid, in place and to another layout."""
    rng = np.random.default_rng(23)
    wide = torch.from_numpy(rng.random((3, 2, max(lens) + 20)).astype(np.float32)).cuda()
    for in_place in (False, True):
        cache, table, _, _ = fill(rng, lens, 3, 32, 16, "bf16")
        weights, before = wide[..., 3:-1].transpose(0, 1), wide.clone()
        want = evicted(cache, table, lens, weights, budget, recent)
        at, _ = on_device(table, lens)
        new = weights
        if not in_place:
            new = torch.full((2, 4, weights.shape[2] + 5), NAN, device="cuda")[:, 1:, 5:]
        got = api.paged_evict(cache, *at, weights, budget, recent, new_weights=new)
        api.poll_status()
        same((cache, *got), want)
        assert torch.equal(wide[..., :3], before[..., :3]) and torch.equal(wide[..., -1:], before[..., -1:])


@pytest.mark.gpu
def test_evict_numbers_of_every_kind():
    """NaN below all, zeros of both signs alike, infinities, subnormals, the largest and smallest."""
    rng = np.random.default_rng(21)
    n, budget = 700, 300
    cache, table, _, _ = fill(rng, [n], 1, 32, 16, "f16")
    kinds = np.array([NAN, -NAN, 0.0, -0.0, np.inf, -np.inf, 1e-45, -1e-45, 3e38, -3e38, 1.0, -1.0, 1.0000001], dtype=np.float32)
    for recent in (0, 30):
        w = kinds[rng.integers(0, len(kinds), (1, 1, n))]
        at, _ = on_device(table, [n])
        weights = torch.from_numpy(w).cuda()
        want = evicted(cache, table, [n], weights, budget, recent)
        got = api.paged_evict(cache, *at, weights, budget, recent)
        api.poll_status()
        same((cache, *got), want)
    for x in (0.0, NAN, np.inf):                                                 # all alike: the first ones stay
        weights = torch.full((1, 1, n), x, device="cuda")
        kept = api.paged_evict(cache, *at, weights, budget, 10)[2]
        assert kept[0, 0].tolist() == [*range(290), *range(690, 700)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,budget", [(20000, 9000), (131072, 131071), (131073, 5), (300001, 123456)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_long_sequences(n, budget, in_place):
    """Clusters of several blocks, and rows that take several rounds."""
    rng = np.random.default_rng(n)
    page, H = 64, 2
    per = -(-n // page)
    table = torch.from_numpy(rng.permutation(2 * per).astype(np.int32)).view(2, per).cuda()
    cache = torch.from_numpy(rng.integers(-2**15, 2**15, (2 * per, 2, H, page, 32), dtype=np.int16)).cuda().view(torch.float16)
    lens = ints([n, n - 1]).cuda()
    weights = torch.from_numpy(np.round(rng.random((2, H, n)) * 1e5).astype(np.float32)).cuda()   # ties
    held = cache.view(torch.int16)[table.long()].permute(0, 2, 3, 1, 4, 5).flatten(3, 4)         # [B, 2, H, slots, D]
    rank = weights.clone()
    rank[1, :, n - 1] = -1
    want = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget].sort(dim=-1).values
    w = weights.gather(2, want)
    new_lens, new, kept = api.paged_evict(cache, table, lens, weights, budget, new_weights=weights if in_place else None, new_lens=lens if in_place else None)
    api.poll_status()
    assert new_lens.tolist() == [min(n, budget), min(n - 1, budget)]
    assert torch.equal(kept.long(), want) and torch.equal(new[..., :budget], w) and not new[..., budget:].any()
    now = cache.view(torch.int16)[table.long()].permute(0, 2, 3, 1, 4, 5).flatten(3, 4)
    moved = held.gather(3, want.view(2, 1, H, budget, 1).expand(-1, 2, -1, -1, 32))
    assert torch.equal(now[:, :, :, :budget], moved) and torch.equal(now[:, :, :, budget:], held[:, :, :, budget:])


@pytest.mark.gpu
def test_evict_with_bad_pages_and_lengths():
    rng = np.random.default_rng(22)
    lens = [60, 60]
    cache, table, _, _ = fill(rng, lens, 1, 64, 16, "bf16")
    weights = torch.from_numpy(rng.random((2, 1, 60)).astype(np.float32)).cuda()
    want = evicted(cache, table, lens, weights, 20, 0)
    page, other = int(table[0, 1]), cache.clone()
    broken = table.clone()
    broken[0, 1] = 99                                                            # tokens 16..31 of the first sequence
    got = api.paged_evict(cache, broken.cuda(), ints(lens).cuda(), weights, 20)
    with pytest.raises(_lib.SdpaError) as e:
        api.poll_status()
    assert e.value.status == INDEX and torch.equal(got[2].cpu(), want[3])
    assert torch.equal(cache[page].view(torch.int16), other[page].view(torch.int16))              # never touched
    for b in table[1].tolist():
        assert torch.equal(cache[b].cpu().view(torch.int16), want[0][b].view(torch.int16))
    for bad in ([-4, 60], [999, 60]):
        got = api.paged_evict(cache, table.cuda(), ints(bad).cuda(), weights, 20)
        with pytest.raises(_lib.SdpaError):
            api.poll_status()
        assert got[0].tolist() == [20 if bad[0] > 0 else 0, 20]


@pytest.mark.gpu
def test_python_refusals():
    cache = api.paged_empty(4, 2, 16, 64, torch.float16)
    q = torch.zeros(2, 4, 3, 64, dtype=torch.float16, device="cuda")
    table, lens = ints([[0], [1]]).cuda(), ints([3, 3]).cuda()
    lse, w = torch.zeros(2, 4, 3, device="cuda"), torch.zeros(2, 2, 16, device="cuda")
    for bad in (lambda: api.paged_weights(q, cache, table, lens, lse[..., :2], w), lambda: api.paged_weights(q, cache, table, lens, lse, w.half()),
                lambda: api.paged_weights(q, cache, table, lens, lse, w[:, :1]), lambda: api.paged_weights(q, cache, table, lens, lse, w[..., ::2]),
                lambda: api.paged_weights(q, cache, table, lens, lse.cpu(), w), lambda: api.paged_weights(q.bfloat16(), cache, table, lens, lse, w),
                lambda: api.paged_evict(cache, table, lens, w, 0), lambda: api.paged_evict(cache, table, lens, w, 4, 5),
                lambda: api.paged_evict(cache, table, lens, w, 4, -1), lambda: api.paged_evict(cache, table, lens, w[:, :1], 4),
                lambda: api.paged_evict(cache, table, lens, w, 4, new_weights=w[..., :8]), lambda: api.paged_evict(cache, table, lens, w, 4, new_lens=lens.long()),
                lambda: api.paged_evict(cache, table, lens, w, 4, kept=torch.zeros(2, 2, 5, dtype=torch.int32, device="cuda")),
                lambda: api.paged_evict(cache[0], table, lens, w, 4), lambda: api.paged_evict(cache, table, lens.cpu(), w, 4)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(_lib.SdpaError):                                          # heads on one address
        api.paged_weights(q, cache, table, lens, lse, w[:, :1].expand(-1, 2, -1))
    with pytest.raises(_lib.SdpaError):                                          # neither in place nor apart
        api.paged_evict(cache, table, lens, w, 4, new_weights=w.view(2, 2, 16).transpose(0, 1))


# ---- together


@pytest.mark.gpu
@pytest.mark.parametrize("G,D,dtype", [(4, 64, "bf16"), (1, 128, "f16")])
def test_a_conversation_in_a_bounded_cache(G, D, dtype):
    """A padded batch of prompts enters in chunks, each with its attention and weights, then decoding
    steps from one captured graph; whenever a sequence may pass the budget it is evicted.  Every step
    is checked against the oracle on what each head has kept."""
    rng = np.random.default_rng(61)
    B, H, page, slots, budget, recent = 3, 2, 16, 160, 100, 20
    scale = 1 / math.sqrt(D)
    table = torch.from_numpy(rng.permutation(B * slots // page).astype(np.int32)).view(B, -1).cuda()
    cache = dirty(B * slots // page, H, page, D, dtype)
    lens = ints([0] * B).cuda()
    weights = torch.full((B, H, slots), NAN, device="cuda")
    held = [[[np.zeros((0, D))] * 2 for _ in range(H)] for _ in range(B)]        # [sequence][head] -> keys, values

    def rows(L):
        return [draw_rows(rng, (B, n, L, D), dtype).cuda() for n in (G * H, H, H)]

    def after(q, k, v, out, lse, old, counts):
        for b in range(B):
            c = counts[b]
            for h in range(H):
                held[b][h] = [np.concatenate([x, as_f64(y)[b, h, q.shape[2] - c:]]) for x, y in zip(held[b][h], (k, v))]
        ks, vs = ([np.stack([held[b][h][x] for h in range(H)]) for b in range(B)] for x in range(2))
        assert lens.tolist() == [k.shape[1] for k in ks]
        check(out, lse, q, ks, vs, scale, True, dtype, counts)
        live = torch.arange(slots, device="cuda") < lens.view(B, 1, 1)
        check_weights(torch.where(live, weights, 0.0), q, ks, vs, lse, torch.where(live, old.nan_to_num(0.0), 0.0), scale, True, counts)

    def evict():
        old, was = weights.cpu().numpy(), lens.tolist()
        kept = api.paged_evict(cache, table, lens, weights, budget, recent, new_lens=lens, new_weights=weights)[2]
        api.poll_status()
        for b in range(B):
            for h in range(H):
                stay = ref.kept(old[b, h], was[b], budget, recent)
                assert kept[b, h, :len(stay)].tolist() == stay
                held[b][h] = [x[stay] for x in held[b][h]]

    for L, counts in ((60, [60, 13, 37]), (60, [60, 60, 1])):
        q, k, v = rows(L)
        new = ints(counts).cuda()
        lens += new
        old = weights.clone()
        api.paged_write(cache, k, v, table, lens, counts=new)
        out, lse = api.paged_attention(q, cache, table, lens, need_lse=True, counts=new)
        api.paged_weights(q, cache, table, lens, lse, weights, counts=new)
        api.poll_status()
        after(q, k, v, out, lse, old, counts)
        evict()

    q, k, v = rows(1)
    old = weights.clone()

    def step():
        lens.add_(1)
        old.copy_(weights)
        api.paged_write(cache, k, v, table, lens)
        out, lse = api.paged_attention(q, cache, table, lens, need_lse=True)
        api.paged_weights(q, cache, table, lens, lse, weights)
        return out, lse

    saved = cache.clone(), lens.clone(), weights.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    for x, y in zip((cache, lens, weights), saved):
        x.copy_(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for n in range(12):
        for x, y in zip((q, k, v), rows(1)):
            x.copy_(y)
        graph.replay()
        api.poll_status()
        after(q, k, v, out, lse, old, [1] * B)
        if n % 4 == 3:
            evict()


@pytest.mark.gpu
def test_eviction_in_a_graph():
    rng = np.random.default_rng(62)
    lens = [90, 40, 77]
    cache, table, _, _ = fill(rng, lens, 2, 32, 16, "f16")
    fresh = cache.clone()
    at, _ = on_device(table, lens)
    w = torch.from_numpy(rng.random((3, 2, 90)).astype(np.float32)).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.paged_evict(cache, *at, w, 50, 5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = api.paged_evict(cache, *at, w, 50, 5)
    for _ in range(3):
        cache.copy_(fresh)
        w.copy_(torch.from_numpy(rng.random((3, 2, 90)).astype(np.float32)))
        want = evicted(cache, table, lens, w, 50, 5)
        graph.replay()
        api.poll_status()
        same((cache, *got), want)
