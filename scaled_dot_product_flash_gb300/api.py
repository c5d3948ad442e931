"""Tensor-level convenience calls over the C ABI (marshalling only).

PyTorch is used here for device memory and streams: outputs are allocated with torch,
their raw device pointers and the current stream's handle are passed to libsdpa.so, and
a non-OK status is raised as ``SdpaError``.  All arithmetic runs in the library.
"""
from __future__ import annotations

import math
import struct

import torch

from . import _lib

DTYPE_CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}

# is_causal values: False/0, True/1 (top-left: key j hidden from query i when j > i) or
# CAUSAL_BOTTOM_RIGHT / "bottom_right" (hidden when j > i + Lkv - Lq; needs Lq <= Lkv).
CAUSAL_NONE, CAUSAL_TOP_LEFT, CAUSAL_BOTTOM_RIGHT = 0, 1, 2


def _causal(c):
    if c is None or c is False:
        return CAUSAL_NONE
    if c is True:
        return CAUSAL_TOP_LEFT
    if c == "bottom_right":
        return CAUSAL_BOTTOM_RIGHT
    if c == "top_left":
        return CAUSAL_TOP_LEFT
    c = int(c)
    if c not in (CAUSAL_NONE, CAUSAL_TOP_LEFT, CAUSAL_BOTTOM_RIGHT):
        raise ValueError(f"is_causal must be False, True or 'bottom_right', not {c}")
    return c


def _check(name, t, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() == 4 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have contiguous rows (stride 1 along D)")
    if t.dim() != 4 and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _layout(t):
    """(batch, head, row) element strides of a [B, H, L, D] tensor: any layout whose rows
    are contiguous, e.g. a [B, L, H, D] buffer seen through .transpose(1, 2)."""
    return (t.stride(0), t.stride(1), t.stride(2))


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _dims(q, k):
    B, Hq, Lq, D = q.shape
    Bk, Hkv, Lkv, Dk = k.shape
    if Bk != B or Dk != D:
        raise ValueError("q and k disagree in batch or head dim")
    return B, Hq, Hkv, Lq, Lkv, D


def _check_sinks(name, t, Hq):
    _check(name, t, torch.float32)
    if t.dim() != 1 or t.numel() != Hq:
        raise ValueError(f"{name} must be a 1-D fp32 tensor of Hq = {Hq} sink logits")


def _mask_layout(shape, strides, elem_size, ptr, Lkv):
    """Whether a 4-D mask view (shape, element strides, element size, address) can be
    passed to the library as it is, and its (batch, head, row) strides with 0 for the
    broadcast (size-1) dimensions.  It can if its keys are contiguous and fill whole
    16-byte pieces and every row starts on a 16-byte boundary."""
    direct = (shape[3] == Lkv and strides[3] == 1 and (Lkv * elem_size) % 16 == 0
              and ptr % 16 == 0
              and all(shape[a] == 1 or (strides[a] * elem_size) % 16 == 0 for a in range(3)))
    return direct, tuple(0 if shape[a] == 1 else strides[a] for a in range(3))


def _mask_arg(attn_mask, q, Lq, Lkv):
    """(Mask struct or None, tensor to keep alive) for an attention mask broadcastable to
    [B, Hq, Lq, Lkv]: boolean (True keeps the key) or floating (added to the scores).

    A mask whose rows are 16-byte aligned, with key stride 1 and a key dimension that
    fills whole 16-byte pieces, is passed as a view (broadcast dimensions get stride 0).
    Otherwise its rows are copied into a buffer with the key dimension padded to 16
    bytes (keeping the broadcast dimensions at size 1); the padding is never read as data.
    """
    if attn_mask is None:
        return None, None
    if not attn_mask.is_cuda or attn_mask.device != q.device:
        raise ValueError("attn_mask must be on the device of q")
    if attn_mask.dim() > 4:
        raise ValueError("attn_mask must have at most 4 dimensions")
    m = attn_mask.reshape((1,) * (4 - attn_mask.dim()) + tuple(attn_mask.shape))
    B, Hq = q.shape[0], q.shape[1]
    for size, want, name in zip(m.shape, (B, Hq, Lq, Lkv), ("batch", "head", "query", "key")):
        if size not in (1, want):
            raise ValueError(f"attn_mask {name} dimension {size} does not broadcast to {want}")
    if m.dtype == torch.bool:
        m, kind = m.view(torch.uint8), _lib.MASK_BOOL
    elif m.is_floating_point():
        m, kind = m.to(q.dtype), _lib.MASK_ADDITIVE
    else:
        raise ValueError("attn_mask must be boolean or floating point")
    es = m.element_size()
    direct, strides = _mask_layout(m.shape, m.stride(), es, m.data_ptr(), Lkv)
    if not direct:
        pad = (Lkv * es + 15) // 16 * 16 // es
        buf = torch.zeros(tuple(m.shape[:3]) + (pad,), device=m.device, dtype=m.dtype)
        buf[..., :Lkv] = m
        m = buf
        _, strides = _mask_layout(m.shape, m.stride(), es, m.data_ptr(), pad)
    return _lib.Mask(m.data_ptr(), kind, *strides), m


def attention_forward(q, k, v, scale=None, is_causal=False, need_lse=True, out=None,
                      lse=None, stream=None, sinks=None, attn_mask=None):
    """out = softmax(scale·q·kᵀ [causal]) · v; also the fp32 logsumexp when need_lse.

    q [B,Hq,Lq,D], k/v [B,Hkv,Lkv,D] CUDA tensors of one dtype (fp32/fp16/bf16), in any
    layout with contiguous rows (e.g. [B,L,H,D] storage seen through .transpose(1, 2));
    the strides go to the library, nothing is copied.  `out` defaults to q's layout.
    ``sinks``: optional fp32 [Hq] sink logits, one extra softmax entry per row of each
    query head with a zero value vector (the lse then includes it).  ``attn_mask``:
    optional mask broadcastable to [B, Hq, Lq, Lkv], boolean (True keeps the key) or
    floating (added to the scaled scores); it combines with ``is_causal``.
    Returns (out, lse or None).
    """
    for n, t in (("q", q), ("k", k), ("v", v)):
        _check(n, t, q.dtype)
    B, Hq, Hkv, Lq, Lkv, D = _dims(q, k)
    if v.shape != k.shape:
        raise ValueError("k and v shapes differ")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)  # same layout as q
    if need_lse and lse is None:
        lse = torch.empty((B, Hq, Lq), device=q.device, dtype=torch.float32)
    if not need_lse:
        lse = None
    _check("out", out, q.dtype)
    if sinks is not None:
        _check_sinks("sinks", sinks, Hq)
    strides = _lib.make_strides(q=_layout(q), k=_layout(k), v=_layout(v), o=_layout(out))
    mask, _keep = _mask_arg(attn_mask, q, Lq, Lkv)
    st = _lib.sdpa_fwd_masked(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                              lse.data_ptr() if lse is not None else None,
                              sinks.data_ptr() if sinks is not None else None, mask,
                              B, Hq, Hkv, Lq, Lkv, D, scale, _causal(is_causal),
                              DTYPE_CODE[q.dtype], strides, _stream(stream))
    if st != _lib.OK:
        raise _lib.SdpaError(st, "sdpa_fwd")
    return out, lse


def workspace_bytes(q, k):
    B, Hq, Hkv, Lq, Lkv, D = _dims(q, k)
    return _lib.sdpa_bwd_workspace_size(B, Hq, Hkv, Lq, Lkv, D, DTYPE_CODE[q.dtype])


def attention_backward(q, k, v, out, dout, lse, scale=None, is_causal=False, workspace=None,
                       dq=None, dk=None, dv=None, stream=None, sinks=None, dsinks=None,
                       attn_mask=None):
    """(dq, dk, dv) of the forward, from its output ``out`` and logsumexp ``lse``.

    ``attn_mask`` must be the forward's mask (it receives no gradient).

    With ``sinks`` (the forward's fp32 [Hq] sink logits), returns (dq, dk, dv, dsinks),
    dsinks being the fp32 [Hq] gradient of the sink logits summed over the batch.
    """
    for n, t in (("q", q), ("k", k), ("v", v), ("out", out), ("dout", dout)):
        _check(n, t, q.dtype)
    _check("lse", lse, torch.float32)
    B, Hq, Hkv, Lq, Lkv, D = _dims(q, k)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = workspace_bytes(q, k)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=q.device, dtype=torch.uint8)
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check(n, t, q.dtype)
    if sinks is not None:
        _check_sinks("sinks", sinks, Hq)
        dsinks = torch.empty_like(sinks) if dsinks is None else dsinks
        _check_sinks("dsinks", dsinks, Hq)
    elif dsinks is not None:
        raise ValueError("dsinks needs sinks")
    strides = _lib.make_strides(q=_layout(q), k=_layout(k), v=_layout(v), o=_layout(out),
                                dout=_layout(dout), dq=_layout(dq), dk=_layout(dk),
                                dv=_layout(dv))
    mask, _keep = _mask_arg(attn_mask, q, Lq, Lkv)
    st = _lib.sdpa_bwd_masked(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                              dout.data_ptr(), lse.data_ptr(),
                              sinks.data_ptr() if sinks is not None else None, mask,
                              dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                              dsinks.data_ptr() if dsinks is not None else None,
                              B, Hq, Hkv, Lq, Lkv, D, scale, _causal(is_causal),
                              DTYPE_CODE[q.dtype], strides, workspace.data_ptr(),
                              workspace.numel(), _stream(stream))
    if st != _lib.OK:
        raise _lib.SdpaError(st, "sdpa_bwd")
    if sinks is not None:
        return dq, dk, dv, dsinks
    return dq, dk, dv


# ---- rotary embedding


# These calls are short on the device, so what a call costs on the host counts: sizes and
# strides go over as packed bytes, and the current stream's handle is asked for directly.
_pack3, _pack6, _pack12 = (struct.Struct(f"{n}q").pack for n in (3, 6, 12))
_pack_cache = struct.Struct("@PiiiiiPqiP").pack  # sdpa_cache_t


def _here(*tensors):
    """Handle of the current stream; every tensor must be on the current device, whose context
    runs the kernels."""
    d = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != d:
            raise ValueError(f"a tensor is on {t.device}, not on the current device, cuda:{d}: "
                             "select its device with torch.cuda.device")
    return torch._C._cuda_getCurrentRawStream(d)


def _rows(name, t, dtype, want=None):
    """Shape and (batch, head, row) strides of a [B, H, L, D] tensor of dtype with contiguous
    rows (and of shape `want`).  Strides of size-1 dimensions, which torch leaves undefined, are
    replaced by D."""
    shape = t.shape
    if len(shape) != 4 or t.dtype is not dtype or not t.is_cuda:
        raise ValueError(f"{name} must be a 4-D [B, H, L, D] CUDA tensor of {dtype}, not "
                         f"{tuple(shape)} of {t.dtype} on {t.device}")
    if want is not None and shape != want:
        raise ValueError(f"{name} must have shape {tuple(want)}, not {tuple(shape)}")
    b, h, r, e = t.stride()
    B, H, L, D = shape
    if e != 1:
        raise ValueError(f"{name} must have contiguous rows (stride 1 along D)")
    return shape, (b if B > 1 else D, h if H > 1 else D, r if L > 1 else D)


def rotary_axes(sections, device="cuda"):
    """int32 [sum(sections)] axis of each pair: the first sections[0] pairs turn by axis 0's
    positions, the next sections[1] by axis 1's, and so on."""
    if any(n < 0 for n in sections) or sum(sections) < 1:
        raise ValueError("sections must be counts of pairs")
    return torch.tensor([a for a, n in enumerate(sections) for _ in range(n)],
                        dtype=torch.int32, device=device)


def _positions(positions, B, L):
    """(axes, strides) of positions [L], [B, L] or [axes, B, L]; B may be 1 for all batches."""
    if positions.dtype not in (torch.int32, torch.int64):
        raise ValueError("positions must be int32 or int64")
    shape, strides = tuple(positions.shape), positions.stride()
    if len(shape) < 3:
        shape, strides = (1,) * (3 - len(shape)) + shape, (0,) * (3 - len(shape)) + strides
    if len(shape) != 3 or shape[1] not in (1, B) or shape[2] != L or shape[0] < 1:
        raise ValueError(f"positions {tuple(positions.shape)} must be [L], [B, L] or [axes, B, L] "
                         f"with L = {L} and B = {B} or 1")
    return shape[0], [0 if n == 1 else s for n, s in zip(shape, strides)]


def _rotary(q, k, positions, inv_freq, axes, adjacent, inverse, q_out, k_out, stream):
    if stream is not None and stream != torch.cuda.current_stream():
        with torch.cuda.stream(stream):  # outputs then belong to that stream
            return _rotary(q, k, positions, inv_freq, axes, adjacent, inverse, q_out, k_out, None)
    dtype = q.dtype
    if dtype not in DTYPE_CODE:
        raise ValueError(f"q has dtype {dtype}, expected fp32, fp16 or bf16")
    shape, qs = _rows("q", q, dtype)
    B, Hq, L, D = shape
    naxes, at = _positions(positions, B, L)
    pairs = inv_freq.shape[0] if inv_freq.dim() == 1 else 0
    if inv_freq.dtype is not torch.float32 or not inv_freq.is_contiguous() or not 2 <= 2 * pairs <= D:
        raise ValueError("inv_freq must be a contiguous 1-D fp32 tensor, one frequency a pair, at "
                         "most D/2")
    if axes is not None and (axes.dtype is not torch.int32 or axes.shape != inv_freq.shape
                             or not axes.is_contiguous()):
        raise ValueError("axes must be a contiguous int32 tensor, one axis for each of inv_freq's "
                         "pairs")
    if q_out is None:
        q_out = torch.empty_like(q)
    _, qos = _rows("q_out", q_out, dtype, shape)
    Hkv, ks, kos, k_ptr, k_out_ptr = 0, (0, 0, 0), (0, 0, 0), None, None
    if k is not None:
        k_shape, ks = _rows("k", k, dtype)
        Hkv = k_shape[1]
        if k_shape[0] != B or k_shape[2] != L or k_shape[3] != D:
            raise ValueError("q and k disagree in batch, rows or head dim")
        if k_out is None:
            k_out = torch.empty_like(k)
        _, kos = _rows("k_out", k_out, dtype, k_shape)
        k_ptr, k_out_ptr = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out needs k")
    st = _lib.sdpa_rotary(
        q.data_ptr(), k_ptr, q_out.data_ptr(), k_out_ptr, positions.data_ptr(),
        64 if positions.dtype is torch.int64 else 32, _pack3(*at), inv_freq.data_ptr(),
        None if axes is None else axes.data_ptr(), naxes, B, Hq, Hkv, L, D, 2 * pairs,
        (_lib.ROTARY_ADJACENT if adjacent else 0) | (_lib.ROTARY_INVERSE if inverse else 0),
        DTYPE_CODE[dtype], _pack12(*qs, *ks, *qos, *kos),
        _here(q, k, positions, inv_freq, axes, q_out, k_out))
    if st != _lib.OK:
        raise _lib.SdpaError(st, "sdpa_rotary")
    return q_out, k_out


def rotary(q, k, positions, inv_freq, axes=None, adjacent=False, q_out=None, k_out=None,
           stream=None):
    """q and k with each pair of elements turned by position·inv_freq; returns both.

    q [B,Hq,L,D] and k [B,Hkv,L,D] (or None) in any layout with contiguous rows; positions
    int32 or int64 [L], [B,L] or [axes,B,L] (B may be 1); inv_freq fp32 [rot/2], rot <= D;
    axes int32 [rot/2] (see ``rotary_axes``): the row of ``positions`` that turns each pair,
    the first for all by default.  Pair p is (p, p + rot/2), or (2p, 2p + 1) when
    ``adjacent``; elements rot and up are copied.  ``q_out=q, k_out=k`` rotates in place.
    """
    return _rotary(q, k, positions, inv_freq, axes, adjacent, False, q_out, k_out, stream)


def rotary_backward(dq_out, dk_out, positions, inv_freq, axes=None, adjacent=False, dq=None,
                    dk=None, stream=None):
    """(dq, dk) of ``rotary`` from the gradients of its outputs: the rotation by the negative
    angles, which also undoes it."""
    return _rotary(dq_out, dk_out, positions, inv_freq, axes, adjacent, True, dq, dk, stream)


# ---- 4-bit paged cache


def cache_empty(num_pages, num_kv_heads, page_size, head_dim, dtype=torch.bfloat16, device="cuda"):
    """Memory of a 4-bit paged cache of keys and values: a tensor of ``dtype`` (fp16 or bf16)
    [num_pages, num_kv_heads, page_size/16, 10·head_dim] whose last dimension is one tile of
    16 tokens, 5 bits an element (``sdpa.h`` has the layout).  Its values mean nothing to
    torch; pages can be copied or moved whole."""
    code = DTYPE_CODE.get(dtype, 0)
    if not _lib.sdpa_cache_page_bytes(page_size, num_kv_heads, head_dim, code) or num_pages < 1:
        raise ValueError("a cache needs fp16 or bf16, a supported head dim and pages of a "
                         "multiple of 16 tokens")
    return torch.empty((num_pages, num_kv_heads, page_size // 16, 10 * head_dim), dtype=dtype,
                       device=device)


def _cache(cache, pages, lens, B):
    """sdpa_cache_t, packed: a cache with one call's page table [B, n] and lengths [B]."""
    dtype = cache.dtype
    if cache.dim() != 4 or not cache.is_cuda or not cache.is_contiguous() or cache.shape[3] % 10:
        raise ValueError("cache must be a contiguous CUDA tensor made by cache_empty")
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError("cache must be fp16 or bf16")
    if pages.dtype is not torch.int32 or pages.dim() != 2 or pages.shape[0] != B or pages.stride(1) != 1:
        raise ValueError(f"pages must be an int32 [{B}, n] tensor with contiguous rows")
    if lens.dtype is not torch.int32 or lens.shape != (B,) or not lens.is_contiguous():
        raise ValueError(f"lens must be a contiguous int32 [{B}] tensor")
    n, H, tiles, width = cache.shape
    entries = pages.shape[1]
    return _pack_cache(cache.data_ptr(), n, 16 * tiles, H, width // 10, DTYPE_CODE[dtype],
                       pages.data_ptr(), pages.stride(0) if B > 1 else entries, entries,
                       lens.data_ptr())


def cache_write(cache, k, v, pages, lens, counts=None, stream=None):
    """Quantises the rows of k and v [B,Hkv,L,D] into the cache, in place.

    pages int32 [B, n]: the pages of each sequence, in order.  lens int32 [B]: tokens of each
    sequence INCLUDING these: row i of L is position lens[b] - L + i, so a padded batch is
    padded on the left, and rows of negative position are not written.  counts int32 [B]: only
    the last counts[b] rows are written.  Pages outside the cache are skipped, a sequence whose
    rows all lie past its table's end is left as it was, and both are reported by ``poll_status``.
    """
    if stream is not None and stream != torch.cuda.current_stream():
        with torch.cuda.stream(stream):
            return cache_write(cache, k, v, pages, lens, counts)
    shape, ks = _rows("k", k, cache.dtype)
    _, vs = _rows("v", v, cache.dtype, shape)
    B, H, L, D = shape
    c = _cache(cache, pages, lens, B)
    if H != cache.shape[1] or 10 * D != cache.shape[3]:
        raise ValueError("k and v must be [B, Hkv, L, D] of the cache's heads and head dim")
    if counts is not None and (counts.dtype is not torch.int32 or counts.shape != (B,)
                               or not counts.is_contiguous()):
        raise ValueError(f"counts must be a contiguous int32 [{B}] tensor")
    st = _lib.sdpa_cache_write(c, k.data_ptr(), v.data_ptr(), _pack6(*ks, *vs),
                               None if counts is None else counts.data_ptr(), B, L,
                               _here(cache, k, v, pages, lens, counts))
    if st != _lib.OK:
        raise _lib.SdpaError(st, "sdpa_cache_write")


def cache_read(cache, pages, lens, rows, k=None, v=None, stream=None):
    """(k, v) [B,Hkv,rows,D]: the last ``rows`` tokens of each sequence as the cache holds
    them, in its dtype.  Row i is position lens[b] - rows + i, 0 where that is negative."""
    if stream is not None and stream != torch.cuda.current_stream():
        with torch.cuda.stream(stream):
            return cache_read(cache, pages, lens, rows, k, v)
    B = lens.numel()
    c = _cache(cache, pages, lens, B)
    shape, dtype = (B, cache.shape[1], rows, cache.shape[3] // 10), cache.dtype
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=cache.device)
    if v is None:
        v = torch.empty(shape, dtype=dtype, device=cache.device)
    _, ks = _rows("k", k, dtype, shape)
    _, vs = _rows("v", v, dtype, shape)
    st = _lib.sdpa_cache_read(c, k.data_ptr(), v.data_ptr(), _pack6(*ks, *vs), B, rows,
                              _here(cache, pages, lens, k, v))
    if st != _lib.OK:
        raise _lib.SdpaError(st, "sdpa_cache_read")
    return k, v


def cache_attention(q, cache, pages, lens, scale=None, is_causal="bottom_right", need_lse=False,
                    out=None, lse=None, sinks=None, max_len=None, workspace=None, stream=None):
    """Attention of q [B,Hq,L,D] over the cached keys and values; returns (out, lse or None).

    pages and lens as in ``cache_write`` (write the rows of this step first).  With the
    default ``is_causal`` query i sees the positions up to its own, lens[b] - L + i; False
    lets it see all lens[b].  A row that sees none gets 0 (lse -inf).  ``sinks`` and the other
    arguments as in ``attention_forward``.  ``max_len`` bounds lens (default: the table's
    width); a tighter bound launches less.  Meant for few rows a KV head; for long chunks
    read the prefix with ``cache_read`` and call ``attention_forward``.
    """
    if stream is not None and stream != torch.cuda.current_stream():
        with torch.cuda.stream(stream):
            return cache_attention(q, cache, pages, lens, scale, is_causal, need_lse, out, lse,
                                   sinks, max_len, workspace)
    dtype = cache.dtype
    shape, qs = _rows("q", q, dtype)
    B, Hq, L, D = shape
    c = _cache(cache, pages, lens, B)
    if 10 * D != cache.shape[3]:
        raise ValueError("q must be [B, Hq, L, D] of the cache's head dim")
    if out is None:
        out = torch.empty_like(q)
    _, os = _rows("out", out, dtype, shape)
    if not need_lse:
        lse = None
    elif lse is None:
        lse = torch.empty((B, Hq, L), device=q.device, dtype=torch.float32)
    elif lse.shape != (B, Hq, L) or lse.dtype is not torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, Hq, L] tensor")
    if sinks is not None:
        _check_sinks("sinks", sinks, Hq)
    max_len = 0 if max_len is None else max(0, min(int(max_len), 2**31 - 1))  # a C int
    need = _lib.sdpa_cache_attn_workspace_size(c, B, Hq, L, max_len)
    if workspace is None and need:
        workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    elif workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    st = _lib.sdpa_cache_attn(
        c, q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
        None if sinks is None else sinks.data_ptr(), _pack6(*qs, *os), B, Hq, L,
        1.0 / math.sqrt(D) if scale is None else float(scale), _causal(is_causal), max_len,
        None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _here(q, cache, pages, lens, out, lse, sinks, workspace))
    if st != _lib.OK:
        raise _lib.SdpaError(st, "sdpa_cache_attn")
    return out, lse


# ---- 16-bit paged cache


_pack2, _pack4 = (struct.Struct(f"{n}q").pack for n in (2, 4))


def paged_empty(num_pages, num_kv_heads, page_size, head_dim, dtype=torch.bfloat16, device="cuda"):
    """Memory of a paged cache of keys and values in 16 bits: a tensor of ``dtype`` (fp16 or
    bf16) [num_pages, 2, num_kv_heads, page_size, head_dim], keys before values."""
    code = DTYPE_CODE.get(dtype, 0)
    if not _lib.sdpa_paged_page_bytes(page_size, num_kv_heads, head_dim, code) or num_pages < 1:
        raise ValueError("a cache needs fp16 or bf16, a supported head dim and pages of a "
                         "multiple of 16 tokens")
    return torch.empty((num_pages, 2, num_kv_heads, page_size, head_dim), dtype=dtype,
                       device=device)


def _paged(cache, pages, lens, B):
    """sdpa_cache_t, packed: a 16-bit cache with one call's page table [B, n] and lengths [B]."""
    dtype = cache.dtype
    if cache.dim() != 5 or not cache.is_cuda or not cache.is_contiguous() or cache.shape[1] != 2:
        raise ValueError("cache must be a contiguous CUDA tensor made by paged_empty")
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError("cache must be fp16 or bf16")
    if pages.dtype is not torch.int32 or pages.dim() != 2 or pages.shape[0] != B or pages.stride(1) != 1:
        raise ValueError(f"pages must be an int32 [{B}, n] tensor with contiguous rows")
    if lens.dtype is not torch.int32 or lens.shape != (B,) or not lens.is_contiguous():
        raise ValueError(f"lens must be a contiguous int32 [{B}] tensor")
    n, _, H, page_size, D = cache.shape
    entries = pages.shape[1]
    return _pack_cache(cache.data_ptr(), n, page_size, H, D, DTYPE_CODE[dtype], pages.data_ptr(),
                       pages.stride(0) if B > 1 else entries, entries, lens.data_ptr())


def _counts(counts, B):
    if counts is None:
        return None
    if counts.dtype is not torch.int32 or counts.shape != (B,) or not counts.is_contiguous():
        raise ValueError(f"counts must be a contiguous int32 [{B}] tensor")
    return counts.data_ptr()


def _weight_rows(name, t, shape):
    """(batch, head) strides of fp32 weights [B, Hkv, slots] with contiguous rows."""
    if t.dtype is not torch.float32 or not t.is_cuda or t.dim() != 3 or (
            tuple(t.shape[:2]) != tuple(shape[:2]) or len(shape) == 3 and t.shape[2] != shape[2]):
        raise ValueError(f"{name} must be an fp32 CUDA tensor {[*shape[:2]]} + [slots], not "
                         f"{tuple(t.shape)} of {t.dtype} on {t.device}")
    b, h, e = t.stride()
    B, H, n = t.shape
    if e != 1 and n > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return (b if B > 1 else H * max(h, n)), (h if H > 1 else n)


def paged_write(cache, k, v, pages, lens, counts=None, stream=None):
    """Copies the rows of k and v [B,Hkv,L,D] into the cache, in place; the other arguments as in
    ``cache_write``."""
    if stream is not None and stream != torch.cuda.current_stream():
        with torch.cuda.stream(stream):
            return paged_write(cache, k, v, pages, lens, counts)
    shape, ks = _rows("k", k, cache.dtype)
    _, vs = _rows("v", v, cache.dtype, shape)
    B, H, L, D = shape
    c = _paged(cache, pages, lens, B)
    if H != cache.shape[2] or D != cache.shape[4]:
        raise ValueError("k and v must be [B, Hkv, L, D] of the cache's heads and head dim")
    st = _lib.sdpa_paged_write(c, k.data_ptr(), v.data_ptr(), _pack6(*ks, *vs), _counts(counts, B),
                               B, L, _here(cache, k, v, pages, lens, counts))
    if st != _lib.OK:
        raise _lib.SdpaError(st, "sdpa_paged_write")


def _max_len(max_len):
    return 0 if max_len is None else max(0, min(int(max_len), 2**31 - 1))  # a C int


def paged_attention(q, cache, pages, lens, scale=None, is_causal="bottom_right", need_lse=False,
                    out=None, lse=None, sinks=None, counts=None, max_len=None, workspace=None,
                    stream=None):
    """Attention of q [B,Hq,L,D] over the keys and values of a 16-bit cache; returns (out, lse or
    None).

    For one token or a few a sequence as for chunks of a prompt (write their rows first).
    counts int32 [B]: only the last counts[b] rows are real; the others of a padded batch give
    0 (lse -inf, or the sink where there is one).  The other arguments as in ``cache_attention``.
    How work is cut over the device goes by max_len, or the width of ``pages``: bound it where the
    table is much wider than the sequences.
    """
    if stream is not None and stream != torch.cuda.current_stream():
        with torch.cuda.stream(stream):
            return paged_attention(q, cache, pages, lens, scale, is_causal, need_lse, out, lse,
                                   sinks, counts, max_len, workspace)
    dtype = cache.dtype
    shape, qs = _rows("q", q, dtype)
    B, Hq, L, D = shape
    c = _paged(cache, pages, lens, B)
    if D != cache.shape[4]:
        raise ValueError("q must be [B, Hq, L, D] of the cache's head dim")
    if out is None:
        out = torch.empty_like(q)
    _, os = _rows("out", out, dtype, shape)
    if not need_lse:
        lse = None
    elif lse is None:
        lse = torch.empty((B, Hq, L), device=q.device, dtype=torch.float32)
    elif lse.shape != (B, Hq, L) or lse.dtype is not torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, Hq, L] tensor")
    if sinks is not None:
        _check_sinks("sinks", sinks, Hq)
    max_len = _max_len(max_len)
    need = _lib.sdpa_paged_attn_workspace_size(c, B, Hq, L, max_len)
    if workspace is None and need:
        workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    elif workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    st = _lib.sdpa_paged_attn(
        c, q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
        None if sinks is None else sinks.data_ptr(), _pack6(*qs, *os), _counts(counts, B), B, Hq, L,
        1.0 / math.sqrt(D) if scale is None else float(scale), _causal(is_causal), max_len,
        None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _here(q, cache, pages, lens, out, lse, sinks, counts, workspace))
    if st != _lib.OK:
        raise _lib.SdpaError(st, "sdpa_paged_attn")
    return out, lse


def paged_weights(q, cache, pages, lens, lse, weights, scale=None, is_causal="bottom_right",
                  counts=None, max_len=None, stream=None):
    """Adds the attention weight of this call's queries to that of the cached tokens, in place;
    returns ``weights``.

    Call it after ``paged_attention`` with the same arguments and the lse that it gave.  weights
    fp32 [B,Hkv,slots]: one sum a token and KV head, over all queries so far and the query heads
    that share the KV head.  The tokens of the call's own rows (the last counts[b], or L) start
    from 0, whatever their slots held.
    """
    if stream is not None and stream != torch.cuda.current_stream():
        with torch.cuda.stream(stream):
            return paged_weights(q, cache, pages, lens, lse, weights, scale, is_causal, counts,
                                 max_len)
    shape, qs = _rows("q", q, cache.dtype)
    B, Hq, L, D = shape
    c = _paged(cache, pages, lens, B)
    if D != cache.shape[4]:
        raise ValueError("q must be [B, Hq, L, D] of the cache's head dim")
    if lse.shape != (B, Hq, L) or lse.dtype is not torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, Hq, L] tensor")
    ws = _weight_rows("weights", weights, (B, cache.shape[2]))
    st = _lib.sdpa_paged_weights(
        c, q.data_ptr(), lse.data_ptr(), weights.data_ptr(), _pack2(*ws), weights.shape[2],
        _pack3(*qs), _counts(counts, B), B, Hq, L,
        1.0 / math.sqrt(D) if scale is None else float(scale), _causal(is_causal),
        _max_len(max_len), _here(q, cache, pages, lens, lse, weights, counts))
    if st != _lib.OK:
        raise _lib.SdpaError(st, "sdpa_paged_weights")
    return weights


def paged_evict(cache, pages, lens, weights, budget, recent=0, new_lens=None, new_weights=None,
                kept=None, stream=None):
    """Shrinks each sequence of more than ``budget`` tokens to that many, in place; returns
    (new_lens, new_weights, kept).

    Each KV head keeps its ``recent`` last tokens and of the others those with the largest
    ``weights`` (fp32 [B,Hkv,slots], see ``paged_weights``; ties go to the earlier token), moved
    together in their order.  new_lens int32 [B] is min(lens, budget), new_weights holds the kept
    tokens' weights and 0 behind them, kept int32 [B,Hkv,budget] the positions that they had (-1
    behind them).  ``new_lens=lens, new_weights=weights`` updates both in place.
    """
    if stream is not None and stream != torch.cuda.current_stream():
        with torch.cuda.stream(stream):
            return paged_evict(cache, pages, lens, weights, budget, recent, new_lens, new_weights,
                               kept)
    B, H, budget = lens.numel(), cache.shape[2] if cache.dim() == 5 else 0, int(budget)
    c = _paged(cache, pages, lens, B)
    ws = _weight_rows("weights", weights, (B, H))
    if not 0 <= recent <= budget or not 1 <= budget < 2**31:
        raise ValueError("budget must be at least 1 and recent within 0 .. budget")
    if new_weights is None:
        new_weights = torch.empty_like(weights)
    ns = _weight_rows("new_weights", new_weights, tuple(weights.shape))
    if new_lens is None:
        new_lens = torch.empty_like(lens)
    elif new_lens.dtype is not torch.int32 or new_lens.shape != (B,) or not new_lens.is_contiguous():
        raise ValueError(f"new_lens must be a contiguous int32 [{B}] tensor")
    if kept is None:
        kept = torch.empty((B, H, budget), dtype=torch.int32, device=cache.device)
    elif kept.dtype is not torch.int32 or kept.shape != (B, H, budget) or not kept.is_contiguous():
        raise ValueError(f"kept must be a contiguous int32 [{B}, {H}, {budget}] tensor")
    st = _lib.sdpa_paged_evict(
        c, weights.data_ptr(), new_weights.data_ptr(), _pack4(*ws, *ns), weights.shape[2],
        new_lens.data_ptr(), kept.data_ptr(), B, budget, int(recent),
        _here(cache, pages, lens, weights, new_lens, new_weights, kept))
    if st != _lib.OK:
        raise _lib.SdpaError(st, "sdpa_paged_evict")
    return new_lens, new_weights, kept


def poll_status(stream=None):
    """Synchronise the stream; raise if a kernel reported a timed-out wait or an index out of
    range."""
    st = _lib.sdpa_poll_status(_stream(stream))
    if st != _lib.OK:
        raise _lib.SdpaError(st, "sdpa_poll_status")


class force_path:
    """Context manager selecting one kernel family (tests and measurements)."""

    def __init__(self, path: int):
        self.path = path

    def __enter__(self):
        st = _lib.sdpa_set_path(self.path)
        if st != _lib.OK:
            raise _lib.SdpaError(st, "sdpa_set_path")
        return self

    def __exit__(self, *exc):
        _lib.sdpa_set_path(_lib.PATH_AUTO)
        return False
