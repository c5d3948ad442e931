// Writing a 4-bit paged cache and reading it back (format in include/sdpa.h).
//
// Bound: HBM for prompts (2·2 bytes an element pair in, 1.25 out, or the reverse), launch
// latency for single tokens.
#include "cache.h"

namespace sdpa {
namespace {

constexpr int kThreads = 256;

// Codes, scale and zero of a group of 32 elements held by 4 neighbouring lanes, 8 each.
// Returns this lane's 8 codes (nibble n = x[n]) and the parameter word (s | z << 16).
// All lanes of the warp call it.
template <typename T>
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], uint32_t& param) {
  float lo = x[0], hi = x[0];
  bool ok = isfinite(x[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
    ok = ok && isfinite(x[e]);
  }
  float bad = ok ? 0.f : 1.f;
#pragma unroll
  for (int off = 1; off <= 2; off <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    bad = fmaxf(bad, __shfl_xor_sync(0xffffffffu, bad, off));
  }
  const float range = __fsub_rn(hi, lo);
  if (bad != 0.f || !isfinite(range)) {
    param = f_to_bits<T>(__int_as_float(0x7fffffff)) << 16;
    return 0;
  }
  const uint32_t sb = f_to_bits<T>(__fdiv_rn(range, 15.f));
  param = sb | (f_to_bits<T>(lo) << 16);
  const float s = bits_to_f<T>(sb);
  uint32_t code = 0;
  if (s > 0.f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float q = fminf(rintf(__fdiv_rn(__fsub_rn(x[e], lo), s)), 15.f);
      code |= (uint32_t)(int)q << (4 * e);
    }
  }
  return code;
}

template <typename T>
__device__ __forceinline__ void load8(float (&x)[8], const T* p) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = bits_to_f<T>(ws[e] & 0xffffu);
    x[2 * e + 1] = bits_to_f<T>(ws[e] >> 16);
  }
}

// One thread an 8-element piece of a key row and of the value row beside it.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(CacheArgs c) {
  using Tl = Tile<D>;
  constexpr int U = D / 8, kRows = kThreads / U;  // pieces a row, rows a block
  const int lrow = threadIdx.x / U, u = threadIdx.x % U;
  const int64_t row = (int64_t)blockIdx.x * kRows + lrow;
  const int64_t rows = (int64_t)c.B * c.Hkv * c.L;
  uint8_t* tile = nullptr;
  int r = 0;
  const T *kp = nullptr, *vp = nullptr;
  if (lrow < kRows && row < rows) {
    const int i = (int)(row % c.L), h = (int)(row / c.L % c.Hkv), b = (int)(row / c.L / c.Hkv);
    const int most = (int)min((int64_t)c.pages_per_seq * c.page_size, (int64_t)0x7fffffff);
    const int count = c.counts ? c.counts[b] : c.L;
    const int pos = cache_len(c, b, most, kKidCacheWrite) - c.L + i;
    if (pos >= 0 && c.L - i <= count) {
      const int page = cache_page(c, b, pos, kKidCacheWrite);
      const int place = pos % c.page_size;
      if (page >= 0) tile = cache_tile<D>(c, page, h, place / kTile);
      r = place % kTile;
      kp = row_ptr<T>(c.k, c.lk, b, h, i) + 8 * u;
      vp = row_ptr<T>(c.v, c.lv, b, h, i) + 8 * u;
    }
  }
  float x[8] = {}, y[8] = {};
  if (tile) {
    load8<T>(x, kp);
    load8<T>(y, vp);
  }
  uint32_t kparam, vparam;
  const uint32_t kc = quantise<T>(x, kparam), vc = quantise<T>(y, vparam);
  if (!tile) return;
  const int j = u / 4, t = u % 4;
  reinterpret_cast<uint32_t*>(tile + Tl::kK)[Tl::k_word(r, t, j)] = kc;
  uint16_t* vh = reinterpret_cast<uint16_t*>(tile + Tl::kV);
  vh[Tl::v_half(r, 2 * t, j)] = (uint16_t)vc;
  vh[Tl::v_half(r, 2 * t + 1, j)] = (uint16_t)(vc >> 16);
  if (t == 0) reinterpret_cast<uint32_t*>(tile + Tl::kKp)[Tl::param(r, j)] = kparam;
  if (t == 1) reinterpret_cast<uint32_t*>(tile + Tl::kVp)[Tl::param(r, j)] = vparam;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, uint32_t code, uint32_t param) {
  const float s = bits_to_f<T>(param & 0xffffu), z = bits_to_f<T>(param >> 16);
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a = fmaf(s, (float)((code >> (8 * e)) & 15u), z), b = fmaf(s, (float)((code >> (8 * e + 4)) & 15u), z);
    w[e] = f_to_bits<T>(a) | (f_to_bits<T>(b) << 16);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheArgs c) {
  using Tl = Tile<D>;
  constexpr int U = D / 8, kRows = kThreads / U;
  const int lrow = threadIdx.x / U, u = threadIdx.x % U;
  const int64_t row = (int64_t)blockIdx.x * kRows + lrow;
  if (lrow >= kRows || row >= (int64_t)c.B * c.Hkv * c.L) return;
  const int i = (int)(row % c.L), h = (int)(row / c.L % c.Hkv), b = (int)(row / c.L / c.Hkv);
  const int most = (int)min((int64_t)c.pages_per_seq * c.page_size, (int64_t)0x7fffffff);
  const int pos = cache_len(c, b, most, kKidCacheRead) - c.L + i;
  uint32_t kc = 0, vc = 0, kparam = 0, vparam = 0;
  if (pos >= 0) {
    const int page = cache_page(c, b, pos, kKidCacheRead);
    if (page >= 0) {
      const int place = pos % c.page_size, r = place % kTile, j = u / 4, t = u % 4;
      const uint8_t* tile = cache_tile<D>(c, page, h, place / kTile);
      kc = reinterpret_cast<const uint32_t*>(tile + Tl::kK)[Tl::k_word(r, t, j)];
      const uint16_t* vh = reinterpret_cast<const uint16_t*>(tile + Tl::kV);
      vc = vh[Tl::v_half(r, 2 * t, j)] | ((uint32_t)vh[Tl::v_half(r, 2 * t + 1, j)] << 16);
      kparam = reinterpret_cast<const uint32_t*>(tile + Tl::kKp)[Tl::param(r, j)];
      vparam = reinterpret_cast<const uint32_t*>(tile + Tl::kVp)[Tl::param(r, j)];
    }
  }
  store8<T>(row_ptr<T>(c.k, c.lk, b, h, i) + 8 * u, kc, kparam);
  store8<T>(row_ptr<T>(c.v, c.lv, b, h, i) + 8 * u, vc, vparam);
}

template <typename T, int D>
cudaError_t launch_t(const CacheArgs& c, bool write, cudaStream_t s) {
  constexpr int kRows = kThreads / (D / 8);
  const unsigned blocks = (unsigned)(((int64_t)c.B * c.Hkv * c.L + kRows - 1) / kRows);
  if (write) cache_write_kernel<T, D><<<blocks, kThreads, 0, s>>>(c);
  else cache_read_kernel<T, D><<<blocks, kThreads, 0, s>>>(c);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_d(const CacheArgs& c, bool write, cudaStream_t s) {
  switch (c.D) {
    case 32: return launch_t<T, 32>(c, write, s);
    case 64: return launch_t<T, 64>(c, write, s);
    case 96: return launch_t<T, 96>(c, write, s);
    case 128: return launch_t<T, 128>(c, write, s);
    case 256: return launch_t<T, 256>(c, write, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_any(const CacheArgs& c, int dtype, bool write, cudaStream_t s) {
  if (dtype == 1) return launch_d<__half>(c, write, s);
  if (dtype == 2) return launch_d<__nv_bfloat16>(c, write, s);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_cache_write(const CacheArgs& c, int dtype, cudaStream_t s) { return launch_any(c, dtype, true, s); }
cudaError_t launch_cache_read(const CacheArgs& c, int dtype, cudaStream_t s) { return launch_any(c, dtype, false, s); }

}  // namespace sdpa
