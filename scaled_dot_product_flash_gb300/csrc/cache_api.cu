// C ABI of the rotary embedding and the 4-bit paged cache: argument checks and launches.
// The operations and every convention are documented in include/sdpa.h.
#include <cmath>
#include <cstring>

#include "cache.h"
#include "host.h"

using namespace sdpa;

namespace {

bool dtype_ok(int dtype) { return dtype == SDPA_F32 || dtype == SDPA_F16 || dtype == SDPA_BF16; }
bool head_dim_ok(int D) { return D == 32 || D == 64 || D == 96 || D == 128 || D == 256; }

// Bytes of the first B rows of a table of int32 with `width` entries a row.
size_t table_bytes(int B, int64_t stride, int width) { return ((size_t)(B - 1) * stride + width) * sizeof(int); }

size_t page_bytes(int page_size, int Hkv, int D) { return (size_t)Hkv * (page_size / kTile) * 20 * D; }

// Checks a cache and the sizes of a call of L rows on it; fills *c but for the rows.
int check_cache(const sdpa_cache_t* cache, int B, int L, CacheArgs* c) {
  if (!cache || B < 1 || L < 1) return SDPA_ERR_INVALID_ARG;
  if (cache->num_pages < 1 || cache->page_size < 1 || cache->Hkv < 1 || cache->D < 1 || cache->pages_per_seq < 1)
    return SDPA_ERR_INVALID_ARG;
  if (cache->page_size % kTile != 0 || cache->pages_stride < cache->pages_per_seq) return SDPA_ERR_INVALID_ARG;
  if (!cache->data || !aligned16(cache->data) || !cache->pages || !aligned4(cache->pages) || !cache->lens || !aligned4(cache->lens))
    return SDPA_ERR_INVALID_ARG;
  if (cache->dtype != SDPA_F16 && cache->dtype != SDPA_BF16) return SDPA_ERR_UNSUPPORTED;
  if (!head_dim_ok(cache->D) || cache->page_size > 65536 || B > 65535 || cache->Hkv > 65535) return SDPA_ERR_UNSUPPORTED;
  // Positions (and a little past them) are 32-bit, offsets in bytes 64-bit.
  if ((double)cache->pages_per_seq * cache->page_size > 1073741824.0 || (double)B * cache->Hkv * L > 1073741824.0) return SDPA_ERR_UNSUPPORTED;
  if (cache->pages_stride > ((int64_t)1 << 40)) return SDPA_ERR_INVALID_ARG;
  std::memset(c, 0, sizeof(*c));
  c->data = static_cast<uint8_t*>(cache->data);
  c->num_pages = cache->num_pages;
  c->page_size = cache->page_size;
  c->Hkv = cache->Hkv;
  c->D = cache->D;
  c->pages = cache->pages;
  c->pages_stride = cache->pages_stride;
  c->pages_per_seq = cache->pages_per_seq;
  c->lens = cache->lens;
  c->B = B;
  c->L = L;
  c->num_sms = sm_count();
  return SDPA_OK;
}

size_t cache_bytes(const CacheArgs& c) { return (size_t)c.num_pages * page_bytes(c.page_size, c.Hkv, c.D); }

// Whether the range [out, out + n) overlaps what describes the cache: its table or lengths.
bool overlaps_tables(const void* out, size_t n, const CacheArgs& c) {
  return overlaps(out, n, c.pages, table_bytes(c.B, c.pages_stride, c.pages_per_seq)) || overlaps(out, n, c.lens, (size_t)c.B * sizeof(int));
}

// A [B, H, L, D] tensor of a call.
struct View {
  const void* p;
  Layout l;
  int H;
  size_t bytes;
};

// Whether two tensors of the same B, L and D share no element.  Besides disjoint ranges this
// knows views of one buffer of tokens (equal batch and row strides) whose heads lie side by
// side in each token, such as q and k inside a fused projection's output: together they must
// be a valid layout of one wide head.
bool apart(const View& x, const View& y, int B, int L, int D, size_t es) {
  if (!overlaps(x.p, x.bytes, y.p, y.bytes)) return true;
  if (x.l.sb != y.l.sb || x.l.sl != y.l.sl) return false;
  const bool x_first = x.p < y.p;
  const View &lo = x_first ? x : y, &hi = x_first ? y : x;
  const int64_t delta = (static_cast<const char*>(hi.p) - static_cast<const char*>(lo.p)) / (int64_t)es;
  const int64_t wide = delta + (hi.H - 1) * hi.l.sh + D;
  if (delta < (lo.H - 1) * lo.l.sh + D || wide > 0x7fffffff) return false;
  Layout unused;
  size_t bytes;
  return check_layout(sdpa_layout_t{lo.l.sb, lo.l.sh, lo.l.sl}, B, 1, L, (int)wide, es, &unused, &bytes);
}

}  // namespace

extern "C" int sdpa_rotary(const void* q, const void* k, void* q_out, void* k_out, const void* positions,
                           int position_bits, const int64_t* position_strides, const float* inv_freq,
                           const int* axes, int naxes, int B, int Hq, int Hkv, int L, int D, int rot,
                           int flags, int dtype, const sdpa_rotary_strides_t* strides, void* stream) {
  if (!k) Hkv = 0;
  if (B < 1 || Hq < 1 || L < 1 || D < 1 || (k && Hkv < 1)) return SDPA_ERR_INVALID_ARG;
  if (!q || !q_out || !positions || !position_strides || !inv_freq || !strides || !k != !k_out) return SDPA_ERR_INVALID_ARG;
  if (rot < 2 || rot > D || rot % 2 != 0 || naxes < 1) return SDPA_ERR_INVALID_ARG;
  if (position_bits != 32 && position_bits != 64) return SDPA_ERR_INVALID_ARG;
  if (flags & ~(SDPA_ROTARY_ADJACENT | SDPA_ROTARY_INVERSE)) return SDPA_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || !head_dim_ok(D)) return SDPA_ERR_UNSUPPORTED;
  if (B > 65535 || Hq > 65535 || Hkv > 65535 || naxes > 65535 || (double)B * L > 2147483647.0) return SDPA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned4(inv_freq) || !aligned4(axes) ||
      reinterpret_cast<uintptr_t>(positions) % (position_bits / 8) != 0)
    return SDPA_ERR_INVALID_ARG;
  RotaryArgs a;
  std::memset(&a, 0, sizeof(a));
  const size_t es = elem_size(dtype);
  size_t qb = 0, kb = 0, qob = 0, kob = 0;
  if (!check_layout(strides->q, B, Hq, L, D, es, &a.lq, &qb) || !check_layout(strides->q_out, B, Hq, L, D, es, &a.lqo, &qob))
    return SDPA_ERR_INVALID_ARG;
  if (k && (!check_layout(strides->k, B, Hkv, L, D, es, &a.lk, &kb) || !check_layout(strides->k_out, B, Hkv, L, D, es, &a.lko, &kob)))
    return SDPA_ERR_INVALID_ARG;
  const int n[3] = {naxes, B, L};
  size_t pb = 1;
  for (int d = 0; d < 3; ++d) {
    if (position_strides[d] < 0 || position_strides[d] > ((int64_t)1 << 40)) return SDPA_ERR_INVALID_ARG;
    pb += (size_t)(n[d] - 1) * position_strides[d];
  }
  pb *= position_bits / 8;
  // In place means the very same elements; any other overlap of an output is refused.
  const auto same = [](const sdpa_layout_t& x, const sdpa_layout_t& y) { return x.batch == y.batch && x.head == y.head && x.row == y.row; };
  const bool q_in_place = q_out == q && same(strides->q, strides->q_out), k_in_place = k && k_out == k && same(strides->k, strides->k_out);
  const View vq{q, a.lq, Hq, qb}, vk{k, a.lk, Hkv, kb}, vqo{q_out, a.lqo, Hq, qob}, vko{k_out, a.lko, Hkv, kob};
  if ((!q_in_place && !apart(vqo, vq, B, L, D, es)) || (k && !k_in_place && !apart(vko, vk, B, L, D, es))) return SDPA_ERR_INVALID_ARG;
  if (k && (!apart(vqo, vk, B, L, D, es) || !apart(vko, vq, B, L, D, es) || !apart(vqo, vko, B, L, D, es))) return SDPA_ERR_INVALID_ARG;
  const void* outs[] = {q_out, k_out};
  const size_t out_bytes[] = {qob, kob};
  const size_t pairs = (size_t)rot / 2 * 4;
  for (int o = 0; o < 2; ++o)
    if (overlaps(outs[o], out_bytes[o], positions, pb) || overlaps(outs[o], out_bytes[o], inv_freq, pairs) || overlaps(outs[o], out_bytes[o], axes, pairs))
      return SDPA_ERR_INVALID_ARG;
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.positions = positions;
  a.pos64 = position_bits == 64;
  a.pos_axis = position_strides[0];
  a.pos_batch = position_strides[1];
  a.pos_row = position_strides[2];
  a.inv_freq = inv_freq;
  a.axes = axes;
  a.naxes = naxes;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.L = L;
  a.D = D;
  a.rot = rot;
  a.adjacent = flags & SDPA_ROTARY_ADJACENT;
  a.inverse = flags & SDPA_ROTARY_INVERSE;
  a.num_sms = sm_count();
  const int st = error_word(&a.err);
  if (st != SDPA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(launch_one(SDPA_KERNEL_ROTARY, s, [&] { return launch_rotary(a, dtype, s); }));
}

extern "C" size_t sdpa_cache_page_bytes(int page_size, int Hkv, int D, int dtype) {
  if (page_size < 1 || page_size % kTile != 0 || page_size > 65536 || Hkv < 1 || Hkv > 65535 || !head_dim_ok(D)) return 0;
  if (dtype != SDPA_F16 && dtype != SDPA_BF16) return 0;
  return page_bytes(page_size, Hkv, D);
}

extern "C" int sdpa_cache_write(const sdpa_cache_t* cache, const void* k, const void* v,
                                const sdpa_layout_t* layouts, const int* counts, int B, int L, void* stream) {
  CacheArgs c;
  int st = check_cache(cache, B, L, &c);
  if (st != SDPA_OK) return st;
  if (!k || !v || !layouts || !aligned16(k) || !aligned16(v) || !aligned4(counts)) return SDPA_ERR_INVALID_ARG;
  size_t kb, vb;
  if (!check_layout(layouts[0], B, c.Hkv, L, c.D, 2, &c.lk, &kb) || !check_layout(layouts[1], B, c.Hkv, L, c.D, 2, &c.lv, &vb))
    return SDPA_ERR_INVALID_ARG;
  const size_t n = cache_bytes(c);
  if (overlaps(c.data, n, k, kb) || overlaps(c.data, n, v, vb) || overlaps(c.data, n, counts, (size_t)B * sizeof(int)) || overlaps_tables(c.data, n, c))
    return SDPA_ERR_INVALID_ARG;
  c.k = const_cast<void*>(k);
  c.v = const_cast<void*>(v);
  c.counts = counts;
  if ((st = error_word(&c.err)) != SDPA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(launch_one(SDPA_KERNEL_CACHE_WRITE, s, [&] { return launch_cache_write(c, cache->dtype, s); }));
}

extern "C" int sdpa_cache_read(const sdpa_cache_t* cache, void* k, void* v, const sdpa_layout_t* layouts, int B,
                               int L, void* stream) {
  CacheArgs c;
  int st = check_cache(cache, B, L, &c);
  if (st != SDPA_OK) return st;
  if (!k || !v || !layouts || !aligned16(k) || !aligned16(v)) return SDPA_ERR_INVALID_ARG;
  size_t kb, vb;
  if (!check_layout(layouts[0], B, c.Hkv, L, c.D, 2, &c.lk, &kb) || !check_layout(layouts[1], B, c.Hkv, L, c.D, 2, &c.lv, &vb))
    return SDPA_ERR_INVALID_ARG;
  const size_t n = cache_bytes(c);
  if (overlaps(k, kb, c.data, n) || overlaps(v, vb, c.data, n) || overlaps(k, kb, v, vb) || overlaps_tables(k, kb, c) || overlaps_tables(v, vb, c))
    return SDPA_ERR_INVALID_ARG;
  c.k = k;
  c.v = v;
  if ((st = error_word(&c.err)) != SDPA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(launch_one(SDPA_KERNEL_CACHE_READ, s, [&] { return launch_cache_read(c, cache->dtype, s); }));
}

namespace {

// Checks the sizes of an attention call and fills them in.
int check_attn(const sdpa_cache_t* cache, int B, int Hq, int Lq, int max_len, CacheAttnArgs* a) {
  std::memset(a, 0, sizeof(*a));
  const int st = check_cache(cache, B, Lq, &a->c);
  if (st != SDPA_OK) return st;
  if (Hq < 1 || Hq % a->c.Hkv != 0) return SDPA_ERR_INVALID_ARG;
  if (Hq > 65535 || (double)B * Hq * Lq > 2147483647.0) return SDPA_ERR_UNSUPPORTED;
  a->Hq = Hq;
  a->G = Hq / a->c.Hkv;
  const int table = a->c.pages_per_seq * a->c.page_size;
  a->max_len = max_len <= 0 || max_len > table ? table : max_len;
  if ((double)a->c.Hkv * cache_attn_row_tiles(*a) > 65535.0) return SDPA_ERR_UNSUPPORTED;
  return SDPA_OK;
}

}  // namespace

extern "C" size_t sdpa_cache_attn_workspace_size(const sdpa_cache_t* cache, int B, int Hq, int Lq, int max_len) {
  CacheAttnArgs a;
  return check_attn(cache, B, Hq, Lq, max_len, &a) == SDPA_OK ? cache_attn_workspace(a) : 0;
}

extern "C" int sdpa_cache_attn(const sdpa_cache_t* cache, const void* q, void* out, float* lse,
                               const float* sinks, const sdpa_layout_t* layouts, int B, int Hq, int Lq,
                               float scale, int is_causal, int max_len, void* workspace,
                               size_t workspace_bytes, void* stream) {
  CacheAttnArgs a;
  int st = check_attn(cache, B, Hq, Lq, max_len, &a);
  if (st != SDPA_OK) return st;
  if (!q || !out || !layouts || !std::isfinite(scale)) return SDPA_ERR_INVALID_ARG;
  if (is_causal < SDPA_CAUSAL_NONE || is_causal > SDPA_CAUSAL_BOTTOM_RIGHT) return SDPA_ERR_INVALID_ARG;
  if (is_causal == SDPA_CAUSAL_TOP_LEFT) return SDPA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(out) || !aligned16(lse) || !aligned4(sinks)) return SDPA_ERR_INVALID_ARG;
  size_t qb, ob;
  if (!check_layout(layouts[0], B, Hq, Lq, a.c.D, 2, &a.lq, &qb) || !check_layout(layouts[1], B, Hq, Lq, a.c.D, 2, &a.lo, &ob))
    return SDPA_ERR_INVALID_ARG;
  const size_t need = cache_attn_workspace(a);
  if (need && (!workspace || workspace_bytes < need)) return SDPA_ERR_WORKSPACE;
  if (need && !aligned16(workspace)) return SDPA_ERR_INVALID_ARG;
  const size_t lb = lse ? (size_t)B * Hq * Lq * sizeof(float) : 0, n = cache_bytes(a.c);
  const void* ins[] = {q, a.c.data, sinks};
  const size_t in_bytes[] = {qb, n, (size_t)Hq * sizeof(float)};
  void* outs[] = {out, lse, workspace};
  const size_t out_bytes[] = {ob, lb, need};
  for (int x = 0; x < 3; ++x) {
    if (overlaps_tables(outs[x], outs[x] ? out_bytes[x] : 0, a.c)) return SDPA_ERR_INVALID_ARG;
    for (int y = 0; y < 3; ++y)
      if (overlaps(outs[x], out_bytes[x], ins[y], in_bytes[y]) || (y > x && overlaps(outs[x], out_bytes[x], outs[y], out_bytes[y])))
        return SDPA_ERR_INVALID_ARG;
  }
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.sinks = sinks;
  a.scale_mant = (float)std::frexp((double)scale * 1.4426950408889634, &a.scale_exp);
  a.causal = is_causal != SDPA_CAUSAL_NONE;
  a.workspace = static_cast<float*>(workspace);
  a.wait_limit_ns = wait_limit_ns();
  if ((st = error_word(&a.c.err)) != SDPA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_one(SDPA_KERNEL_CACHE_ATTN, s, [&] { return launch_cache_attn(a, cache->dtype, s); });
  if (e != cudaSuccess || !need) return status_of(e);
  return status_of(launch_one(SDPA_KERNEL_CACHE_JOIN, s, [&] { return launch_cache_join(a, cache->dtype, s); }));
}
