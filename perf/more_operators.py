"""Measured cases of the 16-bit paged key/value cache: its attention, the attention weight that
its tokens gather, and eviction by that weight.

Operators (``sdpa.h`` and ``scaled_dot_product_flash_gb300.api`` document them in full):

* ``attend``: attention of the last ``L`` queries of each sequence over its cached keys and
  values, bottom-right causal: one token, a few drafted ones, or a chunk of a prompt.  Of a
  padded batch only the last ``counts[b]`` rows are real; the others give 0 (and -inf).
* ``weights``: every cached token's attention weight, summed over the queries of a call and the
  query heads of its KV head: added to what it had, or set for the call's own tokens.
* ``evict``: of each sequence and KV head the ``budget`` tokens with the largest weight stay (the
  last ``recent`` ones in any case; ties go to the earlier token), moved together in their order.
* ``write``: the last ``counts[b]`` rows of each sequence enter their pages.

The cache is a tensor [pages, 2, kv heads, page size, D] of fp16 or bf16, keys before values.
Position j of sequence b lies in page table[b, j // page size], at place j % page size.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
DEVICE = "cuda"
# Of the largest listed cases: products of attention, and bytes of the others.
LARGEST_FLOPS = 1.05e12
LARGEST_BYTES = 5.5e8


def listed():
    return [
        # One short conversation, as many KV heads as query heads: latency.
        {"name": "attend_short_f16", "op": "attend", "type": "f16", "B": 1, "Hq": 8, "Hkv": 8, "L": 1, "D": 64, "page": 16, "max_len": 200, "ragged": False, "sinks": False},
        # Decoding a batch of 32 sequences of 256 to 8192 tokens.
        {"name": "attend_batch_bf16", "op": "attend", "type": "bf16", "B": 32, "Hq": 32, "Hkv": 8, "L": 1, "D": 128, "page": 64, "max_len": 8192, "ragged": True, "sinks": False},
        # Eight drafted tokens checked at once, with sinks (32 rows a KV head).
        {"name": "attend_draft_bf16", "op": "attend", "type": "bf16", "B": 4, "Hq": 32, "Hkv": 8, "L": 8, "D": 128, "page": 64, "max_len": 8192, "ragged": False, "sinks": True},
        # A padded batch of chunks of unequal length, three query heads a KV head, D = 96.
        {"name": "attend_ragged_f16", "op": "attend", "type": "f16", "B": 5, "Hq": 9, "Hkv": 3, "L": 333, "D": 96, "page": 48, "max_len": 1500, "ragged": True, "sinks": False},
        # Prompts of the headline length, in one piece.
        {"name": "attend_prompt_bf16", "op": "attend", "type": "bf16", "B": 2, "Hq": 32, "Hkv": 8, "L": 4096, "D": 128, "page": 64, "max_len": 4096, "ragged": False, "sinks": False},
        # The last chunk of a long document.
        {"name": "attend_chunk_bf16", "op": "attend", "type": "bf16", "B": 1, "Hq": 32, "Hkv": 8, "L": 2048, "D": 128, "page": 128, "max_len": 32768, "ragged": False, "sinks": False},
        # The weights that one step of the decoding batch adds.
        {"name": "weights_batch_bf16", "op": "weights", "type": "bf16", "B": 32, "Hq": 32, "Hkv": 8, "L": 1, "D": 128, "page": 64, "max_len": 8192, "ragged": True, "sinks": False},
        # The weights that a prompt's tokens gather while it enters.
        {"name": "weights_prompt_bf16", "op": "weights", "type": "bf16", "B": 2, "Hq": 32, "Hkv": 8, "L": 4096, "D": 128, "page": 64, "max_len": 4096, "ragged": False, "sinks": False},
        # A decoding batch back from 2304 tokens a sequence to 2048, every 256 steps.
        {"name": "evict_batch_bf16", "op": "evict", "type": "bf16", "B": 32, "Hkv": 8, "D": 128, "page": 64, "max_len": 2304, "ragged": False, "budget": 2048, "recent": 256},
        # A long prompt down to a quarter.
        {"name": "evict_prompt_bf16", "op": "evict", "type": "bf16", "B": 1, "Hkv": 8, "D": 128, "page": 128, "max_len": 32768, "ragged": False, "budget": 8192, "recent": 1024},
        # Decoding: each sequence of a batch of 32 appends one token.
        {"name": "write_token_bf16", "op": "write", "type": "bf16", "B": 32, "Hkv": 8, "L": 1, "D": 128, "page": 16, "max_len": 512, "ragged": True},
        # Prompts of the headline length enter an empty cache.
        {"name": "write_prompt_bf16", "op": "write", "type": "bf16", "B": 2, "Hkv": 8, "L": 4096, "D": 128, "page": 64, "max_len": 4096, "ragged": False},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attend", "attend", "weights", "evict", "write"])
    D = rng.choice([32, 64, 96, 128, 128, 256])
    Hkv, B = rng.randint(1, 8), log(1, 32)
    case = {"op": op, "type": rng.choice(["bf16", "f16"]), "B": B, "Hkv": Hkv, "D": D, "page": 16 * log(1, 16),
            "ragged": rng.random() < 0.7}
    if op == "write":
        room = int(LARGEST_BYTES / 8) // (B * Hkv * D)
        return dict(case, L=max(1, min(log(1, 8192), room)), max_len=max(1, min(log(1, 8192), room)))
    room = int(LARGEST_BYTES / 4) // (B * Hkv * D)
    n = max(1, min(log(1, 65536), room))
    if op == "evict":
        budget = log(1, max(1, n - 1))
        return dict(case, max_len=n, budget=budget, recent=rng.choice([0, rng.randint(0, budget)]))
    G = rng.randint(1, 8)
    L = rng.choice([1, log(1, 16), log(16, 4096)])
    pairs = 1.0e9 / (B * Hkv * G)  # scores of a head at most: 4.3 GB of them in 32 bits
    flops = LARGEST_FLOPS / (4 * B * Hkv * G * D)
    L = max(1, min(L, int(min(pairs, flops) / n)))
    return dict(case, Hq=Hkv * G, L=L, max_len=n, sinks=rng.random() < 0.3)


# ---- sizes


def lengths(case):
    """Tokens of each sequence: all max_len, or evenly spread up to it."""
    B, n = case["B"], case["max_len"]
    return [max(1, n * (b + 1) // B) for b in range(B)] if case["ragged"] else [n] * B


def new_rows(case):
    """How many of a call's L rows are real in each sequence, the rest being padding on the left
    (which order the sequences come in is drawn, and a short one has fewer tokens than that)."""
    B, L = case["B"], case["L"]
    return [max(1, L * (b + 1) // B) for b in range(B)] if case["ragged"] else [L] * B


def work(case):
    D, B, lens = case["D"], case["B"], lengths(case)
    row = case["Hkv"] * D * 2  # bytes of one token's keys (or values)
    if case["op"] == "write":
        new = sum(min(n, c) for n, c in zip(lens, new_rows(case)))
        return {"bytes": 4 * new * row, "flops": 0}
    if case["op"] == "evict":
        budget = case["budget"]
        # Weights read; kept ones, their places and lengths written; keys and values that move:
        # about what lies past the first evicted token, which is near the front.
        moved = sum(budget for n in lens if n > budget)
        heads = case["Hkv"] * 4
        return {"bytes": sum(lens) * heads + 2 * B * budget * heads + 4 * moved * row, "flops": 0}
    Hq, L = case["Hq"], case["L"]
    pairs = seen = 0
    for n, c in zip(lens, new_rows(case)):
        c = min(n, c)
        pairs += c * n - c * (c - 1) // 2  # row i of the last c sees the tokens up to its own
        seen += n
    q = B * Hq * L
    if case["op"] == "attend":
        return {"bytes": 2 * seen * row + 4 * q * D + 4 * q, "flops": 4 * pairs * Hq * D}
    return {"bytes": seen * row + 2 * q * D + 4 * q + 8 * seen * case["Hkv"], "flops": 2 * pairs * Hq * D}


# ---- inputs


def generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def pool(case, seed):
    """A cache with keys and values in it, its page table and the sequences' lengths."""
    rng = np.random.default_rng(seed)
    D, H, page, kind = case["D"], case["Hkv"], case["page"], TYPES[case["type"]]
    lens = rng.permutation(np.array(lengths(case), dtype=np.int64))
    need = -(-lens // page)
    pages = int(need.sum()) + 2
    table = np.full((case["B"], -(-case["max_len"] // page)), -1, dtype=np.int32)
    order = rng.permutation(pages)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    g = generator(seed)
    cache = torch.empty((pages, 2, H, page, D), dtype=kind, device=DEVICE)
    # Keys have a few strong channels, as learned keys do; values are plain.
    offset = 1.5 * torch.randn((H, 1, D), generator=g, device=DEVICE)
    cache[:, 0] = torch.randn((pages, H, page, D), generator=g, device=DEVICE).add_(offset)
    cache[:, 1] = torch.randn((pages, H, page, D), generator=g, device=DEVICE)
    return cache, torch.from_numpy(table).to(DEVICE), torch.from_numpy(lens.astype(np.int32)).to(DEVICE)


def prepare(case, seed):
    cache, table, lens = pool(case, seed)
    state = {"case": case, "cache": cache, "table": table, "lens": lens}
    g = generator(seed + 1)
    B, H, D, kind = case["B"], case["Hkv"], case["D"], TYPES[case["type"]]
    if case["op"] == "evict":
        # Sums of probabilities: most tokens have little, a few much, some none at all.
        w = torch.randn((B, H, case["max_len"]), generator=g, device=DEVICE).mul_(2.0).exp_()
        state["weights"] = w.mul_((torch.rand(w.shape, generator=g, device=DEVICE) > 0.1).float())
        return state
    L = case["L"]
    if case["op"] == "write":
        state["k"], state["v"] = (torch.randn((B, H, L, D), generator=g, device=DEVICE).to(kind) for _ in range(2))
    else:
        state["q"] = torch.randn((B, case["Hq"], L, D), generator=g, device=DEVICE).to(kind)
        state["sinks"] = torch.randn((case["Hq"],), generator=g, device=DEVICE) + 3.0 if case["sinks"] else None
    order = np.random.default_rng(seed + 2).permutation(B)
    state["counts"] = torch.from_numpy(np.array(new_rows(case), dtype=np.int32)[order]).to(DEVICE)
    if case["op"] == "weights":
        state["lse"] = plain_attend(state, False)["lse"]  # the attention's own, of this step
        state["weights"] = torch.rand((B, H, case["max_len"]), generator=g, device=DEVICE)
    return state


# ---- one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return run_own(state)
    if op == "attend":
        return plain_attend(state)
    if op == "weights":
        return plain_weights(state)
    return plain_evict(state) if op == "evict" else plain_write(state)


def run_own(state):
    from scaled_dot_product_flash_gb300 import api

    case, cache, at = state["case"], state["cache"], (state["table"], state["lens"])
    if case["op"] == "attend":
        out, lse = api.paged_attention(state["q"], cache, *at, need_lse=True, sinks=state["sinks"], counts=state["counts"])
        return {"out": out, "lse": lse}
    if case["op"] == "weights":
        return {"weights": api.paged_weights(state["q"], cache, *at, state["lse"], state["weights"], counts=state["counts"])}
    if case["op"] == "evict":
        lens, weights, kept = api.paged_evict(cache, *at, state["weights"], case["budget"], case["recent"])
        return {"cache": cache, "lens": lens, "weights": weights, "kept": kept}
    api.paged_write(cache, state["k"], state["v"], *at, counts=state["counts"])
    return {"cache": cache}


# ---- the plain forms


def place_of(state, position):
    """Page and place of positions [B, ...], whose table entries exist."""
    page = state["case"]["page"]
    b = torch.arange(position.shape[0], device=position.device).view([-1] + [1] * (position.dim() - 1))
    return state["table"].long()[b, position // page], position % page


def plain_rows(state, n, which):
    """fp32 keys (0) or values (1) [B, Hkv, n, D] of the first n positions; those past a
    sequence's end repeat its last one."""
    position = torch.arange(n, device=DEVICE).minimum(state["lens"].long().unsqueeze(1) - 1)
    page, place = place_of(state, position)
    return state["cache"][page, which, :, place].transpose(1, 2).float()


def plain_scores(state, n):
    """Scaled scores [B, Hkv, G·L, n], -inf where a row does not see a token."""
    case, q = state["case"], state["q"].float()
    B, Hq, L, D = q.shape
    scores = q.view(B, case["Hkv"], -1, D) @ plain_rows(state, n, 0).transpose(2, 3)
    scores /= math.sqrt(D)
    lens = state["lens"].long().view(B, 1, 1, 1)
    row = torch.arange(L, device=DEVICE).repeat(Hq // case["Hkv"]).view(1, 1, -1, 1)
    real = row >= L - state["counts"].long().view(B, 1, 1, 1)
    hidden = (torch.arange(n, device=DEVICE) > lens - L + row) | ~real
    return scores.masked_fill_(hidden, -math.inf)


def plain_attend(state, values=True):
    case = state["case"]
    B, Hq, L, D = state["q"].shape
    scores = plain_scores(state, case["max_len"])
    top = scores.amax(-1, keepdim=True)
    if state["sinks"] is not None:
        sink = state["sinks"].view(1, case["Hkv"], -1, 1).repeat_interleave(L, 2)
        top = top.maximum(sink)
    top = torch.where(top == -math.inf, 0.0, top)
    weight = scores.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    if state["sinks"] is not None:
        total = total + (sink - top).exp()
    lse = (top + total.log()).view(B, Hq, L)
    if not values:
        return {"lse": lse}
    out = torch.where(total > 0, (weight @ plain_rows(state, case["max_len"], 1)) / total, 0.0)
    return {"out": out.view(B, Hq, L, D).to(state["q"].dtype), "lse": lse}


def plain_weights(state):
    n = state["case"]["max_len"]
    lse = state["lse"].flatten(1).view(state["lse"].shape[0], state["case"]["Hkv"], -1, 1)
    p = plain_scores(state, n).sub_(torch.where(lse == -math.inf, 0.0, lse)).exp_()
    gain = p.sum(2)
    lens = state["lens"].long().view(-1, 1, 1)
    slot = torch.arange(n, device=DEVICE)
    old = slot < lens - state["counts"].long().view(-1, 1, 1)
    weights = state["weights"]
    weights.copy_(torch.where(slot < lens, torch.where(old, weights, 0.0) + gain, weights))
    return {"weights": weights}


def plain_evict(state):
    case, cache, weights = state["case"], state["cache"], state["weights"]
    budget, n = case["budget"], weights.shape[2]
    lens = state["lens"].long().view(-1, 1, 1)
    slot = torch.arange(n, device=DEVICE)
    rank = weights.masked_fill(slot >= lens - case["recent"], math.inf).masked_fill_(slot >= lens, -math.inf)
    short = min(budget, n)
    kept = rank.sort(dim=-1, descending=True, stable=True).indices[..., :short].sort(dim=-1).values
    new_lens = lens.clamp(max=budget)
    there = torch.arange(short, device=DEVICE) < new_lens
    new_weights = torch.zeros_like(weights)
    new_weights[..., :short] = weights.gather(2, kept) * there
    b, h, r = (there & (lens > budget)).expand_as(kept).nonzero(as_tuple=True)  # the tokens of shortened sequences
    page, place = place_of(state, kept)
    source = page[b, h, r], place[b, h, r]
    page, place = place_of(state, torch.arange(short, device=DEVICE).minimum(lens.flatten(1) - 1))
    to = page[b, r], place[b, r]
    cache[to[0], :, h, to[1]] = cache[source[0], :, h, source[1]]
    places = torch.full((*weights.shape[:2], budget), -1, dtype=torch.int32, device=DEVICE)
    places[..., :short] = torch.where(there, kept, -1)
    return {"cache": cache, "lens": new_lens.view(-1).to(torch.int32), "weights": new_weights, "kept": places}


def plain_write(state):
    L, cache = state["case"]["L"], state["cache"]
    row = torch.arange(L, device=DEVICE)
    position = state["lens"].long().unsqueeze(1) - L + row
    real = (position >= 0) & (row >= L - state["counts"].long().unsqueeze(1))
    page, place = place_of(state, position.clamp(min=0))
    new = torch.stack((state["k"], state["v"])).permute(1, 3, 0, 2, 4)  # [B, L, 2, Hkv, D]
    cache[page[real], :, :, place[real]] = new[real]
    return {"cache": cache}


# ---- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    B, H, D = case["B"], case["Hkv"], case["D"]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    cache = s["cache"]

    def held(b, which):
        """Keys or values [Hkv, length, D] of sequence b."""
        pages = torch.tensor([p for p in table[b] if p >= 0], device=DEVICE)
        return cache[pages, which].transpose(0, 1).reshape(H, -1, D)[:, :lens[b]].double()

    if case["op"] in ("write", "evict"):
        want = cache.double()

        def put(b, h, which, first, rows):
            """Rows [n, D] from position `first` on; all heads where h is None, rows [Hkv, n, D]."""
            n, page, done = rows.shape[-2], case["page"], 0
            while done < n:
                at, place = divmod(first + done, page)
                step = min(page - place, n - done)
                want[table[b][at], which, slice(None) if h is None else h, place:place + step] = rows[..., done:done + step, :]
                done += step

    if case["op"] == "write":
        for b, c in enumerate(s["counts"].tolist()):
            c = min(c, lens[b])
            for which, x in enumerate((s["k"], s["v"])):
                put(b, None, which, lens[b] - c, x[b, :, case["L"] - c:].double())
        return {"cache": want}
    if case["op"] == "evict":
        budget = case["budget"]
        kept, weights = np.full((B, H, budget), -1, dtype=np.int32), np.zeros(s["weights"].shape)
        w = s["weights"].double().cpu().numpy()
        for b, n in enumerate(lens):
            rows = [held(b, 0), held(b, 1)] if n > budget else None
            for h in range(H):
                stay = np.arange(n)
                if n > budget:
                    old = n - case["recent"]
                    best = np.lexsort((np.arange(old), -w[b, h, :old]))[:budget - case["recent"]]
                    stay = np.concatenate([np.sort(best), np.arange(old, n)])
                    for which in range(2):
                        put(b, h, which, 0, rows[which][h, torch.from_numpy(stay).to(DEVICE)])
                kept[b, h, :len(stay)] = stay
                weights[b, h, :len(stay)] = w[b, h, stay]
        return {"cache": want, "lens": torch.tensor([min(n, budget) for n in lens], dtype=torch.int32, device=DEVICE),
                "weights": torch.from_numpy(weights).to(DEVICE), "kept": torch.from_numpy(kept).to(DEVICE)}
    q, L, G = s["q"].double(), case["L"], case["Hq"] // H
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=DEVICE)
    out, weights = torch.zeros_like(q), s["weights"].double() if case["op"] == "weights" else None
    for b, c in enumerate(s["counts"].tolist()):
        c, n = min(c, lens[b]), lens[b]
        k, v = held(b, 0), held(b, 1)
        i, j = torch.arange(n - c, n, device=DEVICE).view(1, -1, 1), torch.arange(n, device=DEVICE)
        if weights is not None:
            weights[b, :, n - min(s["counts"].tolist()[b], n):n] = 0.0
        for h in range(H):
            group = slice(h * G, h * G + G)
            x = torch.einsum("gid,jd->gij", q[b, group, L - c:], k[h]) * D ** -0.5
            x = x.masked_fill(j > i, -math.inf)
            if weights is not None:
                weights[b, h, :n] += torch.exp(x - s["lse"][b, group, L - c:, None].double()).sum((0, 1))
                continue
            total = torch.logsumexp(x, -1)
            if s["sinks"] is not None:
                total = torch.logaddexp(total, s["sinks"][group].double().view(-1, 1).expand_as(total))
            lse[b, group, L - c:] = total
            out[b, group, L - c:] = torch.einsum("gij,jd->gid", torch.exp(x - total.unsqueeze(-1)), v[h])
    if weights is not None:
        return {"weights": weights}
    if s["sinks"] is not None:  # a row that sees no token rests on its sink
        lse = torch.where(lse == -math.inf, s["sinks"].double().view(1, -1, 1).expand_as(lse), lse)
    return {"out": out, "lse": lse}
