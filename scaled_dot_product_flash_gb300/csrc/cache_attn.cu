// Attention over a 4-bit paged cache (format and conventions in include/sdpa.h).
//
// One warp a query row: 32 keys at a time, a key a lane for the scores, the running maximum
// and sum of the softmax, then the head dimension over the lanes for the values.
#include "cache.h"

namespace sdpa {
namespace {

constexpr int kWarps = 4;

template <typename T, int D>
__device__ __forceinline__ float cached(const uint8_t* tile, bool value, int r, int d) {
  using Tl = Tile<D>;
  const int j = d / kGroup, e = d % kGroup;
  uint32_t code, param;
  if (value) {
    code = (reinterpret_cast<const uint16_t*>(tile + Tl::kV)[Tl::v_half(r, e / 4, j)] >> (4 * (e % 4))) & 15u;
    param = reinterpret_cast<const uint32_t*>(tile + Tl::kVp)[Tl::param(r, j)];
  } else {
    code = (reinterpret_cast<const uint32_t*>(tile + Tl::kK)[Tl::k_word(r, e / 8, j)] >> (4 * (e % 8))) & 15u;
    param = reinterpret_cast<const uint32_t*>(tile + Tl::kKp)[Tl::param(r, j)];
  }
  return fmaf(bits_to_f<T>(param & 0xffffu), (float)code, bits_to_f<T>(param >> 16));
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) cache_attn_kernel(CacheAttnArgs a) {
  __shared__ float qs[kWarps][D];
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t row = (int64_t)blockIdx.x * kWarps + warp;
  if (row >= (int64_t)c.B * a.Hq * c.L) return;
  const int i = (int)(row % c.L), hq = (int)(row / c.L % a.Hq), b = (int)(row / c.L / a.Hq), h = hq / a.G;
  const T* q = row_ptr<T>(a.q, a.lq, b, hq, i);
  for (int d = lane; d < D; d += 32) qs[warp][d] = Elem<T>::to_f(q[d]);
  __syncwarp();
  const int len = cache_len(c, b, a.max_len, kKidCacheAttn);
  const int end = a.causal ? len - c.L + i + 1 : len;
  float m = minus_inf(), l = 0.f, o[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
  for (int j0 = 0; j0 < end; j0 += 32) {
    const int pos = j0 + lane;
    const uint8_t* tile = nullptr;
    if (pos < end) {
      const int page = cache_page(c, b, pos, kKidCacheAttn);
      if (page >= 0) tile = cache_tile<D>(c, page, h, pos % c.page_size / kTile);
    }
    float s = minus_inf();
    if (tile) {
      float acc = 0.f;
      for (int d = 0; d < D; ++d) acc = fmaf(qs[warp][d], cached<T, D>(tile, false, pos % kTile, d), acc);
      s = acc * a.scale_log2;
    }
    float top = s;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float m_new = fmaxf(m, top), ref = m_new == minus_inf() ? 0.f : m_new;
    const float alpha = exp2f(m - ref), p = exp2f(s - ref);
    float sum = p;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    l = l * alpha + sum;
    m = m_new;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] *= alpha;
    for (int jj = 0; jj < 32; ++jj) {
      const uint8_t* t = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(tile), jj));
      const float pj = __shfl_sync(0xffffffffu, p, jj);
      if (!t) continue;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) o[e] = fmaf(pj, cached<T, D>(t, true, (j0 + jj) % kTile, lane + 32 * e), o[e]);
    }
  }
  const float fold = fold_sink(a.sinks, hq, m, l);
  T* out = row_ptr<T>(a.out, a.lo, b, hq, i);
#pragma unroll
  for (int e = 0; e < D / 32; ++e) out[lane + 32 * e] = Elem<T>::from_f(l == 0.f ? 0.f : o[e] * fold / l);
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? minus_inf() : (m + log2f(l)) * kLn2;
}

template <typename T, int D>
cudaError_t attn_t(const CacheAttnArgs& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.c.B * a.Hq * a.c.L;
  cache_attn_kernel<T, D><<<(unsigned)((rows + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t attn_d(const CacheAttnArgs& a, cudaStream_t s) {
  switch (a.c.D) {
    case 32: return attn_t<T, 32>(a, s);
    case 64: return attn_t<T, 64>(a, s);
    case 96: return attn_t<T, 96>(a, s);
    case 128: return attn_t<T, 128>(a, s);
    case 256: return attn_t<T, 256>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

size_t cache_attn_workspace(const CacheAttnArgs&) { return 0; }

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int dtype, cudaStream_t s) {
  if (dtype == 1) return attn_d<__half>(a, s);
  if (dtype == 2) return attn_d<__nv_bfloat16>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
