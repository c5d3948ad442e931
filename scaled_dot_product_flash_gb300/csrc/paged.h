// Internal parameters, launchers and device helpers of the 16-bit paged cache (its layout and
// conventions are documented in include/sdpa.h).
#pragma once

#include <atomic>

#include "cache.h"
#include "tc_common.cuh"

namespace sdpa {

// Attention over the cache, and the weights that its tokens gather (c.counts: real rows).
struct PagedArgs {
  CacheArgs c;
  const void* q;
  void* out;
  float* lse;           // attention: written, nullable; weights: read
  const float* sinks;   // nullable
  Layout lq, lo;
  int Hq, G;
  float scale_log2;     // scale·log2(e)
  int causal;
  int max_len;          // longest sequence, in tokens
  float* workspace;
  float* weights;       // [B][Hkv][slots]
  int64_t w_batch, w_head;
  uint64_t wait_limit_ns;
};
bool paged_attn_launchable(const PagedArgs& a);   // whether its blocks fit a grid
size_t paged_attn_workspace(const PagedArgs& a);  // 0: one kernel does it all
cudaError_t launch_paged_attn(const PagedArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_paged_join(const PagedArgs& a, int dtype, cudaStream_t s);  // after it, with a workspace
cudaError_t launch_paged_weights(const PagedArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_paged_write(const CacheArgs& a, cudaStream_t s);

// How attention's first `rows` queries of each sequence are cut: into `splits` chunks of `chunk` tokens,
// whose partial results are joined.  They lie in the workspace as [B][Hq][rows][splits] rows of D
// elements, unnormalised, then as many pairs (maximum, sum).
struct Cut {
  int chunk, splits, rows;
};

// Attention's form for many rows a KV head.
bool paged_chunk_takes(const PagedArgs& a);
Cut paged_chunk_cut(const PagedArgs& a);
int64_t paged_chunk_blocks(const PagedArgs& a);
cudaError_t launch_paged_chunk(const PagedArgs& a, int dtype, cudaStream_t s);
// And the weights'.
bool paged_gain_takes(const PagedArgs& a);
cudaError_t launch_paged_gain(const PagedArgs& a, int dtype, cudaStream_t s);

// Division of numbers below 2^31 by a divisor that a call fixes: with l = ceil(log2 d) and
// m = floor(2^(31+l) / d) + 1, n / d = floor(n·m / 2^(31+l)), since m·d exceeds 2^(31+l) by d <= 2^l
// at most and n < 2^31.
struct Divider {
  uint32_t m;
  int shift;  // l - 1; a divisor of 1 has shift -1
  __device__ __forceinline__ int operator()(int n) const { return shift < 0 ? n : (int)(__umulhi((uint32_t)n, m) >> shift); }
};
inline Divider divider(int d) {
  int l = 0;
  while (((int64_t)1 << l) < d) ++l;
  return Divider{(uint32_t)(((uint64_t)1 << (31 + l)) / d + 1), l - 1};
}

// Sets a kernel's shared-memory limit once on each device.
template <typename K>
cudaError_t allow_smem(K* kern, int bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (ready.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

struct EvictArgs {
  CacheArgs c;
  const float* weights;
  float* new_weights;
  int64_t w_batch, w_head, nw_batch, nw_head;
  int* kept;      // [B][Hkv][budget]
  int* new_lens;  // [B]
  int budget, recent, slots;  // slots: entries of a row of weights
  Divider by_page;            // by page_size
};
cudaError_t launch_paged_select(const EvictArgs& a, cudaStream_t s);
cudaError_t launch_paged_move(const EvictArgs& a, cudaStream_t s);

// 4-D tensor map over a cache of 16-bit pages: box of `rows` tokens of 64 elements at
// (x = element, y = place in the page, h = Hkv·(0 keys, 1 values) + head, b = page).
inline bool make_tmap_pages(CUtensorMap* map, const CacheArgs& c, int rows) {
  const int64_t head = (int64_t)c.page_size * c.D;
  return make_tmap_4d(map, c.data, c.D, c.page_size, 2 * c.Hkv, c.num_pages, Layout{2 * c.Hkv * head, head, c.D}, rows);
}

// What the rows of a call see.  Row i (0 <= i < L) of a sequence of len tokens has position
// len - L + i; it is real if it is among the last `count` rows.
struct Rows {
  int len, first, L;  // first: the first real row
  int causal;
  // Tokens [0, limit) are seen by row i.
  __device__ __forceinline__ int limit(int i) const {
    if (i < first) return 0;
    return causal ? max(0, len - L + i + 1) : len;
  }
};
__device__ __forceinline__ Rows rows_of(const CacheArgs& c, int b, int causal, int most, unsigned kid) {
  Rows r;
  r.len = cache_len(c, b, most, kid);
  const int count = c.counts ? min(max(c.counts[b], 0), c.L) : c.L;
  r.first = c.L - count;
  r.L = c.L;
  r.causal = causal;
  return r;
}

// Index of a partial result.
__device__ __forceinline__ int64_t part_of(const Cut& cut, int b, int Hq, int hq, int i, int split) {
  return (((int64_t)b * Hq + hq) * cut.rows + i) * cut.splits + split;
}
// Where the pairs of the partial results begin.
__device__ __forceinline__ float* part_stats(const PagedArgs& a, const Cut& cut) {
  return a.workspace + (int64_t)a.c.B * a.Hq * cut.rows * cut.splits * a.c.D;
}

// Element offset of a row of a page: which = 0 keys, 1 values.
__device__ __forceinline__ int64_t paged_row(const CacheArgs& c, int page, int which, int h, int place) {
  return ((((int64_t)page * 2 + which) * c.Hkv + h) * c.page_size + place) * c.D;
}

// P = 2^(c·s − base) meets V in T.  A row's base follows its scores lazily, since O has to be rescaled with
// it: it rises where a tile's maximum passes the one it was set by by 2^8.  bf16 has fp32's exponents and takes
// that maximum itself as the base.  fp16 ends below 2^16 and loses bits under 2^-14, so there the base lies 7
// below it, and it falls again where a tile's weights all lie under 2^-7, as they do behind a token that
// outweighs the others.  A weight is off by 2^-25·2^base then, apart from its rounding to the type's bits: by at
// most 2^-32 of the row's largest and 2^-18 of its tile's largest.  (Sums of 16 more bits per weight, for few rows, do not
// help against the end of the exponents.)
template <typename T>
constexpr bool kNarrow = std::is_same<T, __half>::value;
constexpr float kRescale = 8.f, kFall = 7.f, kBias = 7.f;
constexpr float kExact = 4194304.f;  // 2^22: below it a base can lie 7 below a maximum with P still under 2^16

template <typename T>
__device__ __forceinline__ float bias_of(float x) { return kNarrow<T> && fabsf(x) < kExact ? kBias : 0.f; }
// The base for a largest score of top.
template <typename T>
__device__ __forceinline__ float base_of(float top) { return top - bias_of<T>(top); }
// The score past which it rises.
template <typename T>
__device__ __forceinline__ float base_high(float base) { return base + (kRescale + bias_of<T>(base)); }
// (What lies 2^60 below the row's sum l adds nothing; O stays far from fp32's end.)
__device__ __forceinline__ bool base_falls(float base, float top, float l) { return top < base - kFall && l * tc::ex2(base - top) < 0x1p60f; }

// For columns [d, d + N) of an output o of query (hq, i) of KV head h over the tokens [from, to) of
// sequence b, some of which came out NaN without a reason in the row's scores, since a product meets
// every value of a tile, under a weight of 0 too.  Those with a value among the tokens that is not finite are
// infinite or NaN accordingly; the others, where the value belongs to a token that the row does not
// see, are Σ exp2(c·q·k_j − M)·v_j once more, product by product in fp32, one thread a row.
// A value that is not finite in the last token of 60 queries over 16384 tokens costs 20 ms so in bf16 and at
// D = 256, 78 in fp16 at D = 128, element by element, and one at the end of 16384 for one or two queries 0.4.  What
// the loops of paged_chunk.cu take depends on what this function looks like: pieces of 8 cost fp16 prompts 3% and
// bf16 ones nothing; the sums in registers, 4 ms here, 7%; warp-level MMAs, 1 to 2 ms here, 25%.
template <typename T, int D, int N>
__device__ __noinline__ void mend_columns(const PagedArgs& a, int b, int h, int hq, int i, int d, int from, int to, float M, float* o) {
  const CacheArgs& c = a.c;
  const T* q = row_ptr<T>(a.q, a.lq, b, hq, i);
  const T* data = reinterpret_cast<const T*>(c.data);
  uint32_t open = 0;  // columns whose NaN is not explained yet
  for (int y = 0; y < N; ++y)
    if (o[y] != o[y]) {
      open |= 1u << y;
      o[y] = 0.f;
    }
  uint32_t nan = 0;
  for (int j = from; j < to && (open & ~nan); ++j) {
    const int page = c.pages[b * c.pages_stride + j / c.page_size], place = j % c.page_size;
    if ((unsigned)page >= (unsigned)c.num_pages) continue;
    const T* v = data + paged_row(c, page, 1, h, place) + d;
    for (uint32_t left = open & ~nan; left; left &= left - 1) {
      const int y = __ffs(left) - 1;
      const float z = Elem<T>::to_f(v[y]);
      if (fabsf(z) < __builtin_huge_valf()) continue;
      o[y] += z;  // (inf - inf is NaN)
      if (o[y] != o[y]) nan |= 1u << y;
    }
  }
  for (int y = 0; y < N; ++y)
    if (o[y] != 0.f) open &= ~(1u << y);
  if (!open) return;
  constexpr int kStep = D == 256 || (!kNarrow<T> && N == 32) ? 4 : 1;  // tokens at a time, of one page
  for (int j = from; j < to; j += kStep) {
    const int page = c.pages[b * c.pages_stride + j / c.page_size], place = j % c.page_size;
    if ((unsigned)page >= (unsigned)c.num_pages) continue;
    const T* k = data + paged_row(c, page, 0, h, place);
    const T* v = data + paged_row(c, page, 1, h, place) + d;
    float s[kStep] = {};
    if constexpr (kNarrow<T> && N == 32 && D < 256) {
      for (int y = 0; y < D; ++y) s[0] = fmaf(Elem<T>::to_f(q[y]), Elem<T>::to_f(k[y]), s[0]);
    } else {
#pragma unroll 2
      for (int y = 0; y < D; y += 8) {
        const uint4 x4 = *reinterpret_cast<const uint4*>(q + y);
        const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
        for (int n = 0; n < kStep; ++n) {
          const uint4 z4 = *reinterpret_cast<const uint4*>(k + n * D + y);
          const uint32_t z[4] = {z4.x, z4.y, z4.z, z4.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float x0, x1, z0, z1;
            tc::unpack2<T>(x[u], x0, x1);
            tc::unpack2<T>(z[u], z0, z1);
            s[n] = fmaf(x0, z0, s[n]);
            s[n] = fmaf(x1, z1, s[n]);
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < kStep; ++n) {
      if (j + n >= to) break;
      const float p = tc::ex2(s[n] * a.scale_log2 - M);
      for (int y = 0; y < N; ++y)
        if (open >> y & 1u) o[y] = fmaf(p, Elem<T>::to_f(v[n * D + y]), o[y]);
    }
  }
}

}  // namespace sdpa
