"""Measured cases of the 4-bit paged key/value cache and of the rotary embedding.

Operators (``sdpa.h`` and ``scaled_dot_product_flash_gb300.api`` document them in full):

* ``write``: the last rows of each sequence are quantised to 4 bits into their pages; a
  pass reads the rows just written back, since they are the values the cache holds.
* ``read``: the last rows of each sequence as the cache holds them, in the element type.
* ``attend``: attention of the last ``L`` queries of each sequence over its cached keys and
  values, bottom-right causal.
* ``rotary``: rotation of queries and keys by their positions (one or several axes), and
  with ``grad`` the gradients too.

The cache is a tensor [pages, kv heads, page size / 16, 10·D] of the element type (fp16 or
bf16).  The last dimension is one tile of 16 tokens, 20·D bytes.  A row of D elements is
split into D/32 groups of 32; a group has a scale s and a zero z (its minimum), both in the
element type, and an element is z + s·code with a code of 0..15.  With NG = D/32 groups,
W = min(NG, 4) and group j = W·jb + w, a tile holds

  K codes  [row half][jb][g = row % 8][t][w] 32-bit words; nibble n is element 32j + 8t + n
  V codes  [row half][jb][g][t][w] words; the low 16 bits are row 8·half + 2t, the high ones
           row 8·half + 2t + 1; nibble n of those is element 32j + 4g + n
  K params [jb][row][w] pairs (s, z), then V params the same
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEVICE = "cuda"
LARGEST = 3.3e8  # bytes of a pass of the largest listed case


def listed():
    return [
        # One new token a sequence: positions far into a long context, 32 query and 8 KV heads.
        {"name": "rotary_token_bf16", "op": "rotary", "type": "bf16", "B": 4, "Hq": 32, "Hkv": 8, "L": 1, "D": 128, "rot": 128, "axes": 1, "adjacent": False, "far": 1000000, "grad": False},
        # A training step at the headline attention's shape, time/height/width axes, gradients.
        {"name": "rotary_train_bf16", "op": "rotary", "type": "bf16", "B": 2, "Hq": 32, "Hkv": 8, "L": 4096, "D": 128, "rot": 128, "axes": 3, "adjacent": False, "far": 4096, "grad": True},
        # Images of 24 x 24 patches and a class token, fp32, adjacent pairs, a part of D rotated.
        {"name": "rotary_image_f32", "op": "rotary", "type": "f32", "B": 8, "Hq": 8, "Hkv": 8, "L": 577, "D": 64, "rot": 48, "axes": 2, "adjacent": True, "far": 24, "grad": True},
        # Decoding: each sequence of a batch of 32 appends one token.
        {"name": "write_token_bf16", "op": "write", "type": "bf16", "B": 32, "Hkv": 8, "L": 1, "D": 128, "page": 16, "max_len": 512, "ragged": True},
        # Prompts of the headline length enter an empty cache.
        {"name": "write_prompt_bf16", "op": "write", "type": "bf16", "B": 2, "Hkv": 8, "L": 4096, "D": 128, "page": 64, "max_len": 4096, "ragged": False},
        # A padded batch of chunks of unequal length, odd sizes, D = 96.
        {"name": "write_chunk_f16", "op": "write", "type": "f16", "B": 5, "Hkv": 3, "L": 333, "D": 96, "page": 48, "max_len": 1500, "ragged": True},
        # The prefix of a chunked prompt, read back for the tiled attention kernels.
        {"name": "read_prefix_bf16", "op": "read", "type": "bf16", "B": 4, "Hkv": 8, "L": 8192, "D": 128, "page": 64, "max_len": 8192, "ragged": True},
        # A sliding window of a small model.
        {"name": "read_window_f16", "op": "read", "type": "f16", "B": 7, "Hkv": 2, "L": 255, "D": 64, "page": 16, "max_len": 2000, "ragged": True},
        # One short conversation, as many KV heads as query heads: latency.
        {"name": "attend_short_f16", "op": "attend", "type": "f16", "B": 1, "Hq": 8, "Hkv": 8, "L": 1, "D": 64, "page": 16, "max_len": 200, "ragged": False, "sinks": False},
        # Decoding a batch of 32 sequences of 256 to 8192 tokens.
        {"name": "attend_batch_bf16", "op": "attend", "type": "bf16", "B": 32, "Hq": 32, "Hkv": 8, "L": 1, "D": 128, "page": 64, "max_len": 8192, "ragged": True, "sinks": False},
        # One sequence with a long context.
        {"name": "attend_long_bf16", "op": "attend", "type": "bf16", "B": 1, "Hq": 32, "Hkv": 8, "L": 1, "D": 128, "page": 128, "max_len": 131072, "ragged": False, "sinks": False},
        # Eight drafted tokens checked at once, with sinks (32 rows a KV head).
        {"name": "attend_draft_bf16", "op": "attend", "type": "bf16", "B": 4, "Hq": 32, "Hkv": 8, "L": 8, "D": 128, "page": 64, "max_len": 8192, "ragged": True, "sinks": True},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rotary", "write", "read", "attend"])
    D = rng.choice([32, 64, 96, 128, 128, 256])
    Hkv = rng.randint(1, 8)
    if op == "rotary":
        B, L, Hq = log(1, 8), log(1, 4096), Hkv * rng.randint(1, 4)
        case = {"op": op, "type": rng.choice(["bf16", "f16", "f32"]), "B": B, "Hq": Hq, "Hkv": Hkv, "L": L, "D": D,
                "rot": rng.choice([D, 2 * rng.randint(D // 8, D // 2)]), "axes": rng.randint(1, 4),
                "adjacent": rng.random() < 0.5, "far": log(16, 1000000), "grad": rng.random() < 0.5}
        return dict(case, L=max(1, min(L, int(LARGEST * L / work(case)["bytes"]))))
    B = log(1, 32)
    case = {"op": op, "type": rng.choice(["bf16", "f16"]), "B": B, "Hkv": Hkv, "D": D, "page": 16 * log(1, 16),
            "ragged": rng.random() < 0.7}
    if op == "attend":
        Hq, L = Hkv * rng.randint(1, 8), log(1, 16)
        room = min(int(1.3e8) // (B * Hkv * D), int(2.6e9) // (4 * B * Hq * L * D))
        return dict(case, Hq=Hq, L=L, max_len=max(1, min(log(1, 32768), room)), sinks=rng.random() < 0.3)
    room = int(LARGEST / 11) // (B * Hkv * D)
    return dict(case, L=max(1, min(log(1, 8192), room)), max_len=max(1, min(log(1, 8192), room)))


# ---- sizes


def lengths(case):
    """Tokens of each sequence: all max_len, or evenly spread up to it."""
    B, n = case["B"], case["max_len"]
    return [max(1, n * (b + 1) // B) for b in range(B)] if case["ragged"] else [n] * B


def new_rows(case):
    """How many of the L rows of a write are real, the rest being padding on the left."""
    B, L = case["B"], case["L"]
    return [L * (b + 1) // B if L > 1 else 1 for b in range(B)] if case["ragged"] else [L] * B


def work(case):
    D, L, B = case["D"], case["L"], case["B"]
    size = TYPES[case["type"]].itemsize
    if case["op"] == "rotary":
        rows = B * L * (case["Hq"] + case["Hkv"])
        passes = 2 if case["grad"] else 1
        return {"bytes": passes * (2 * rows * D * size + 4 * B * L * case["axes"]), "flops": passes * 3 * rows * case["rot"]}
    lens, row = lengths(case), case["Hkv"] * D  # elements of one token's keys (or values)
    if case["op"] == "attend":
        q = B * case["Hq"] * L * D
        return {"bytes": sum(lens) * row * 1.25 + 2 * q * size + (4 * B * case["Hq"] * L), "flops": 4 * sum(lens) * case["Hq"] * L * D}
    held = sum(min(n, L) for n in lens)
    values = 2 * B * L * row * size
    if case["op"] == "read":
        return {"bytes": held * row * 1.25 + values, "flops": 2 * 2 * held * row}
    new = sum(min(n, c, L) for n, c in zip(lens, new_rows(case)))
    return {"bytes": new * row * (2 * size + 1.25) + held * row * 1.25 + values, "flops": 2 * 4 * new * row + 2 * 2 * held * row}


# ---- inputs


def generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def codes_of(x):
    """The definition of the format, in fp32 steps: z = min, s = (max - min) / 15 rounded to the
    element type, code = round((x - z) / s) to even, within 0..15 (0 where s is 0)."""
    kind = x.dtype
    x = x.float().unflatten(-1, (-1, 32))
    z, high = x.amin(-1), x.amax(-1)
    s = ((high - z) / 15.0).to(kind)
    step = s.float().unsqueeze(-1)
    code = torch.where(step > 0, (x - z.unsqueeze(-1)) / step, 0.0).round().clamp(0, 15)
    return code.to(torch.uint8).flatten(-2), s, z.to(kind)


def pool(case, seed):
    """A pool of pages with keys and values in it: codes [pages, Hkv, tiles, 16, D], scales and
    zeros [pages, Hkv, tiles, 16, D/32] of both, and the page table and lengths."""
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
    shape = (pages, H, page // 16, 16, D)
    # Keys have a few strong channels, as learned keys do; values are plain.
    offset = 1.5 * torch.randn((H, 1, 1, D), generator=g, device=DEVICE)
    k = codes_of(torch.randn(shape, generator=g, device=DEVICE).add_(offset).to(kind))
    v = codes_of(torch.randn(shape, generator=g, device=DEVICE).to(kind))
    return k, v, torch.from_numpy(table).to(DEVICE), torch.from_numpy(lens.astype(np.int32)).to(DEVICE)


def packed(k, v):
    """The cache tensor of codes, scales and zeros (the layout in the module's docstring)."""
    (kc, ks, kz), (vc, vs, vz) = k, v
    lead, D = kc.shape[:-2], kc.shape[-1]
    n = len(lead)
    NG = D // 32
    W = min(NG, 4)
    JB = NG // W
    a = list(range(n))

    def order(x, dims):
        return x.permute(a + [n + d for d in dims])

    # K: (half, g, jb, w, t, byte, nibble) -> (half, jb, g, t, w, byte, nibble)
    x = order(kc.reshape(*lead, 2, 8, JB, W, 4, 4, 2), (0, 2, 1, 4, 3, 5, 6))
    kb = (x[..., 0] | (x[..., 1] << 4)).reshape(*lead, 8 * D)
    # V: (half, t, parity, jb, w, g, byte, nibble) -> (half, jb, g, t, w, parity, byte, nibble)
    x = order(vc.reshape(*lead, 2, 4, 2, JB, W, 8, 2, 2), (0, 3, 5, 1, 4, 2, 6, 7))
    vb = (x[..., 0] | (x[..., 1] << 4)).reshape(*lead, 8 * D)
    params = []
    for s, z in ((ks, kz), (vs, vz)):
        x = torch.stack([s, z], -1).reshape(*lead, 16, JB, W, 2)
        params.append(order(x, (1, 0, 2, 3)).reshape(*lead, D))
    return torch.cat([kb.view(ks.dtype), vb.view(ks.dtype)] + params, -1)


def frequencies(case):
    """fp32 [rot/2] angular frequencies and the axis of each pair (contiguous sections)."""
    n = case["rot"] // 2
    inv = torch.from_numpy((10000.0 ** (-np.arange(n, dtype=np.float64) / n)).astype(np.float32)).to(DEVICE)
    axes = torch.from_numpy((np.arange(n) * case["axes"] // n).astype(np.int32)).to(DEVICE)
    return inv, axes


def rotary_inputs(case, seed):
    g = generator(seed)
    kind, B, L, D = TYPES[case["type"]], case["B"], case["L"], case["D"]
    rows = {}
    for name, H in (("q", case["Hq"]), ("k", case["Hkv"])):
        for grad in ([name, "d" + name] if case["grad"] else [name]):
            rows[grad] = torch.randn((B, H, L, D), generator=g, device=DEVICE).to(kind)
    if case["axes"] == 1:  # text: consecutive positions from some place in the context
        start = torch.randint(0, case["far"] + 1, (1, B, 1), generator=g, device=DEVICE)
        positions = start + torch.arange(L, device=DEVICE)
    else:
        positions = torch.randint(0, case["far"] + 1, (case["axes"], B, L), generator=g, device=DEVICE)
    inv, axes = frequencies(case)
    return dict(rows, positions=positions.to(torch.int32), inv=inv, axes=axes)


def prepare(case, seed):
    if case["op"] == "rotary":
        return dict(rotary_inputs(case, seed), case=case)
    k, v, table, lens = pool(case, seed)
    state = {"case": case, "cache": packed(k, v), "table": table, "lens": lens}
    del k, v
    g = generator(seed + 1)
    B, H, L, D, kind = case["B"], case["Hkv"], case["L"], case["D"], TYPES[case["type"]]
    if case["op"] == "attend":
        state["q"] = torch.randn((B, case["Hq"], L, D), generator=g, device=DEVICE).to(kind)
        state["sinks"] = torch.randn((case["Hq"],), generator=g, device=DEVICE) + 3.0 if case["sinks"] else None
    if case["op"] == "write":
        state["k"], state["v"] = (torch.randn((B, H, L, D), generator=g, device=DEVICE).to(kind) for _ in range(2))
        state["counts"] = torch.tensor(new_rows(case), dtype=torch.int32, device=DEVICE)
    return state


# ---- one pass


def run(state):
    if own:
        return run_own(state)
    case = state["case"]
    if case["op"] == "rotary":
        return plain_rotary(state)
    if case["op"] == "write":
        plain_write(state)
    if case["op"] in ("write", "read"):
        k, v, _ = plain_rows(state["cache"], state["table"], state["lens"], case["L"])
        return {"k": k.to(state["cache"].dtype), "v": v.to(state["cache"].dtype)}
    return plain_attend(state)


def run_own(state):
    from scaled_dot_product_flash_gb300 import api

    case = state["case"]
    if case["op"] == "rotary":
        how = (state["positions"], state["inv"], state["axes"], case["adjacent"])
        q, k = api.rotary(state["q"], state["k"], *how)
        if not case["grad"]:
            return {"q": q, "k": k}
        dq, dk = api.rotary_backward(state["dq"], state["dk"], *how)
        return {"q": q, "k": k, "dq": dq, "dk": dk}
    if case["op"] == "attend":
        out, lse = api.cache_attention(state["q"], state["cache"], state["table"], state["lens"], need_lse=True,
                                       sinks=state["sinks"])
        return {"out": out, "lse": lse}
    if case["op"] == "write":
        api.cache_write(state["cache"], state["k"], state["v"], state["table"], state["lens"], state["counts"])
    k, v = api.cache_read(state["cache"], state["table"], state["lens"], case["L"])
    return {"k": k, "v": v}


# ---- the plain forms


def plain_rotary(state):
    case = state["case"]
    half = case["rot"] // 2
    angle = state["positions"].double()[state["axes"].long()].permute(1, 2, 0) * state["inv"].double()
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)

    def turn(x, sin):
        x32, rot = x.float(), case["rot"]
        if case["adjacent"]:
            a, b = x32[..., 0:rot:2], x32[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x32[..., :half], x32[..., half:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x32[..., rot:]], -1).to(x.dtype)

    out = {"q": turn(state["q"], sin), "k": turn(state["k"], sin)}
    if case["grad"]:
        out.update(dq=turn(state["dq"], -sin), dk=turn(state["dk"], -sin))
    return out


def plain_tiles(tiles):
    """fp32 keys and values [..., 16, D] of cache tiles [..., 10·D]."""
    D, lead = tiles.shape[-1] // 10, tiles.shape[:-1]
    n = len(lead)
    NG = D // 32
    W = min(NG, 4)
    JB = NG // W
    a = list(range(n))
    raw = tiles.contiguous().view(torch.uint8)

    def nibbles(x):
        return torch.stack([x & 15, x >> 4], -1)

    kc = nibbles(raw[..., :8 * D].reshape(*lead, 2, JB, 8, 4, W, 4))
    kc = kc.permute(a + [n + d for d in (0, 2, 1, 4, 3, 5, 6)]).reshape(*lead, 16, NG, 32)
    vc = nibbles(raw[..., 8 * D:16 * D].reshape(*lead, 2, JB, 8, 4, W, 2, 2))
    vc = vc.permute(a + [n + d for d in (0, 3, 5, 1, 4, 2, 6, 7)]).reshape(*lead, 16, NG, 32)
    out = []
    for code, at in ((kc, 8 * D), (vc, 9 * D)):
        p = tiles[..., at:at + D].reshape(*lead, JB, 16, W, 2).float()
        p = p.permute(a + [n + d for d in (1, 0, 2, 3)]).reshape(*lead, 16, NG, 2)
        out.append((p[..., 1:] + p[..., :1] * code.float()).flatten(-2))
    return out


def plain_rows(cache, table, lens, L):
    """fp32 keys and values [B, Hkv, L, D] of each sequence's last L positions (0 where the
    position is negative), and which of them there are [B, L]."""
    per_page = cache.shape[2]
    n = lens.long().unsqueeze(1)
    first = torch.div(n - L, 16, rounding_mode="floor")
    tile = first + torch.arange(-(-L // 16) + 1, device=cache.device)
    tile = tile.clamp(min=0).minimum((n - 1).clamp(min=0) // 16)
    page = table.long().gather(1, tile // per_page).clamp(min=0)
    k, v = plain_tiles(cache[page, :, tile % per_page])
    position = n - L + torch.arange(L, device=cache.device)
    there = position >= 0
    # Row of the gathered tiles that holds each position: its tile's place, then its place in it.
    place = (torch.div(position, 16, rounding_mode="floor") - first) * 16 + position.remainder(16)
    out = []
    for x in (k, v):
        x = x.transpose(1, 2).flatten(2, 3)
        x = x.gather(2, place[:, None, :, None].expand(-1, x.shape[1], -1, x.shape[3]))
        out.append(torch.where(there[:, None, :, None], x, 0.0))
    return out[0], out[1], there


def plain_offsets(D, device):
    """Byte offsets inside a tile of the D/2 bytes of each of its 16 rows, for K and for V, and
    element offsets of the D/32 (s, z) pairs."""
    NG = D // 32
    W = min(NG, 4)
    row = torch.arange(16, device=device).unsqueeze(1)
    i = torch.arange(D // 2, device=device)  # byte of the row in element order
    j, t, byte = i // 16, i % 16 // 4, i % 4
    k = ((((row // 8 * (NG // W) + j // W) * 8 + row % 8) * 4 + t) * W + j % W) * 4 + byte
    g, byte = i % 16 // 2, i % 2
    v = 8 * D + ((((row // 8 * (NG // W) + j // W) * 8 + g) * 4 + row % 8 // 2) * W + j % W) * 4 + row % 2 * 2 + byte
    j = torch.arange(NG, device=device)
    return k, v, 8 * D + ((j // W * 16 + row) * W + j % W) * 2


def plain_write(state):
    case, cache = state["case"], state["cache"]
    B, H, L, D = state["k"].shape
    per_page = cache.shape[2]
    position = state["lens"].long().unsqueeze(1) - L + torch.arange(L, device=cache.device)
    real = (position >= 0) & (torch.arange(L, device=cache.device) >= L - state["counts"].long().unsqueeze(1))
    b, i = real.nonzero(as_tuple=True)
    position = position[b, i]
    page = state["table"].long()[b, position // case["page"]]
    head = torch.arange(H, device=cache.device)
    tile = (page.unsqueeze(1) * H + head) * per_page + (position % case["page"] // 16).unsqueeze(1)  # [rows, H]
    row = position % 16
    k_at, v_at, p_at = plain_offsets(D, cache.device)
    raw, flat = cache.view(torch.uint8).view(-1), cache.view(-1)
    for x, at, more in ((state["k"], k_at, 0), (state["v"], v_at, D)):
        code, s, z = codes_of(x.transpose(1, 2)[b, i])  # [rows, H, D]
        raw[tile.unsqueeze(2) * (20 * D) + at[row].unsqueeze(1)] = code[..., 0::2] | (code[..., 1::2] << 4)
        place = tile.unsqueeze(2) * (10 * D) + more + p_at[row].unsqueeze(1)
        flat[place] = s
        flat[place + 1] = z


def plain_attend(state):
    case, q = state["case"], state["q"].float()
    B, Hq, L, D = q.shape
    n = case["max_len"]
    k, v, there = plain_rows(state["cache"], state["table"], state["lens"], n)
    q = q.view(B, k.shape[1], -1, D)  # the query heads of a KV head, and their rows
    scores = (q @ k.transpose(2, 3)) / math.sqrt(D)
    row = torch.arange(L, device=q.device).repeat(q.shape[2] // L)
    seen = torch.arange(n, device=q.device) - n <= row.unsqueeze(1) - L
    scores = torch.where(there[:, None, None] & seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    if state["sinks"] is not None:
        sink = state["sinks"].view(1, k.shape[1], -1, 1).repeat_interleave(L, 2)
        top = top.maximum(sink)
    top = torch.where(top == -math.inf, 0.0, top)
    weight = (scores - top).exp()
    total = weight.sum(-1, keepdim=True)
    if state["sinks"] is not None:
        total = total + (sink - top).exp()
    out = torch.where(total > 0, (weight @ v) / total, 0.0)
    lse = top + total.log()
    return {"out": out.view(B, Hq, L, D).to(state["q"].dtype), "lse": lse.view(B, Hq, L)}


# ---- the definitions in 64 bits


def exact(case, seed):
    if case["op"] == "rotary":
        return exact_rotary(case, rotary_inputs(case, seed))
    B, H, L, D, kind = case["B"], case["Hkv"], case["L"], case["D"], TYPES[case["type"]]
    (kc, ks, kz), (vc, vs, vz), table, lens = pool(case, seed)
    table, lens = table.tolist(), lens.tolist()
    g = generator(seed + 1)

    def held(b):
        """Keys and values [Hkv, length, D] of sequence b."""
        pages = torch.tensor([p for p in table[b] if p >= 0], device=DEVICE)
        got = []
        for c, s, z in ((kc, ks, kz), (vc, vs, vz)):
            x = c[pages].double().unflatten(-1, (-1, 32)) * s[pages].double().unsqueeze(-1) + z[pages].double().unsqueeze(-1)
            got.append(x.flatten(-2).transpose(0, 1).reshape(H, -1, D)[:, :lens[b]])
        return got

    if case["op"] == "attend":
        q = torch.randn((B, case["Hq"], L, D), generator=g, device=DEVICE).to(kind).double()
        sinks = (torch.randn((case["Hq"],), generator=g, device=DEVICE) + 3.0).double() if case["sinks"] else None
        out, lse = torch.zeros_like(q), torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=DEVICE)
        for b in range(B):
            k, v = held(b)
            G = case["Hq"] // H
            s = torch.einsum("hgid,hjd->hgij", q[b].unflatten(0, (H, G)), k) / D ** 0.5
            i, j = torch.arange(L, device=DEVICE).unsqueeze(1), torch.arange(lens[b], device=DEVICE)
            s = s.masked_fill(j > i + lens[b] - L, -math.inf).flatten(0, 1)
            if sinks is not None:  # a last key with a value of zero
                s = torch.cat([s, sinks.view(-1, 1, 1).expand(-1, L, 1)], -1)
            lse[b] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[b].unsqueeze(-1)).nan_to_num(0.0)[..., :lens[b]]
            out[b] = torch.einsum("hgij,hjd->hgid", p.unflatten(0, (H, G)), v).flatten(0, 1)
        return {"out": out, "lse": lse}
    want = {}
    new = [torch.randn((B, H, L, D), generator=g, device=DEVICE).to(kind).double() for _ in range(2)] if case["op"] == "write" else None
    rows = [torch.zeros((B, H, L, D), dtype=torch.float64, device=DEVICE) for _ in range(2)]
    for b in range(B):
        have = min(lens[b], L)
        for x, old in zip(rows, held(b)):
            x[b, :, L - have:] = old[:, lens[b] - have:]
        if new is not None:
            real = min(new_rows(case)[b], have)
            for x, y in zip(rows, new):
                if real:
                    group = y[b, :, L - real:].unflatten(-1, (-1, 32))
                    low, high = group.min(-1, keepdim=True).values, group.max(-1, keepdim=True).values
                    step = ((high - low) / 15).to(kind).double()
                    code = torch.where(step > 0, (group - low) / step, 0.0).round().clamp(0, 15)
                    x[b, :, L - real:] = (low + step * code).flatten(-2)
    want["k"], want["v"] = rows
    return want


def exact_rotary(case, x):
    """Each pair as a complex number times e^(i·angle)."""
    rot = case["rot"]
    angle = torch.stack([x["positions"][int(a)].double() * f for a, f in zip(x["axes"].tolist(), x["inv"].double())], -1)
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    out = {}
    for name in [n for n in ("q", "k", "dq", "dk") if n in x]:
        y = x[name].double().clone()
        pair = y[..., :rot].unflatten(-1, (-1, 2)) if case["adjacent"] else y[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous()) * (turn.conj() if name.startswith("d") else turn)
        pair = torch.view_as_real(z)
        y[..., :rot] = pair.flatten(-2) if case["adjacent"] else pair.transpose(-1, -2).flatten(-2)
        out[name] = y
    return out
