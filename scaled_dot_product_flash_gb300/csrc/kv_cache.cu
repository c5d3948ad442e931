// Writing a 4-bit paged cache and reading it back (format in include/sdpa.h).
//
// A warp takes the keys or the values of half a tile (8 tokens of one head), in the order in
// which the tile is stored: lane (g, t) = (lane / 4, lane % 4) has row g of the half and of each
// group elements 8t..8t+7, so that inputs and outputs move in 16-byte pieces, 64 contiguous bytes a row and group; K words
// leave as 512 contiguous bytes, and V words are the same words after an 8 x 8 transpose of
// their halves (movmatrix), since a V half-word is 4 elements of one row and its word two
// neighbouring rows.  Rows of a tile that a call does not touch are masked at the stores: a K
// word belongs to one row, of a V word only the half is stored then.
//
// Bound: HBM for prompts (4 bytes in and 1.25 out for an element of K and of V, or the
// reverse), launch latency for single tokens.
#include "cache.h"

namespace sdpa {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Eight 16-bit elements as fp32.
template <typename T>
__device__ __forceinline__ void unpack8(float (&x)[8], const uint4& w) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = bits_to_f<T>(ws[e] & 0xffffu);
    x[2 * e + 1] = bits_to_f<T>(ws[e] >> 16);
  }
}

// Codes, scale and zero of a group of 32 elements held by the 4 lanes of a quad, 8 each.
// Returns this lane's 8 codes (nibble n = x[n]) and the parameter word (s | z << 16).
template <typename T>
__device__ __forceinline__ uint32_t quantise(const uint4& in, uint32_t& param) {
  constexpr float kInf = __builtin_huge_valf();
  float x[8];
  unpack8<T>(x, in);
  float lo = x[0], hi = x[0];
  bool fine = fabsf(x[0]) < kInf;
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
    fine = fine && fabsf(x[e]) < kInf;
  }
  if (!fine) hi = kInf;
#pragma unroll
  for (int off = 1; off <= 2; off <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
  }
  const float range = __fsub_rn(hi, lo);
  if (!(range < kInf)) {
    param = f_to_bits<T>(__int_as_float(0x7fffffff)) << 16;
    return 0;
  }
  const uint32_t sb = f_to_bits<T>(__fdiv_rn(range, 15.f));
  param = sb | (f_to_bits<T>(lo) << 16);
  const float s = bits_to_f<T>(sb);
  // The quotient rounded correctly from the reciprocal rounded correctly, one residual step
  // (Markstein 1990), so that ties fall as the definition has them.  Scales near the end of
  // fp32's range, where that would underflow, divide.
  float c[8];
  if (s > 0x1p-100f) {
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = __fsub_rn(x[e], lo), q = __fmul_rn(d, inv);
      c[e] = fmaf(fmaf(-q, s, d), inv, q);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = s > 0.f ? __fdiv_rn(__fsub_rn(x[e], lo), s) : 0.f;
  }
  constexpr float kRound = 12582912.f;  // 1.5·2^23: adding it rounds to an integer, ties to even
#pragma unroll
  for (int e = 0; e < 8; ++e) c[e] = __fsub_rn(__fadd_rn(fminf(c[e], 15.f), kRound), kRound);
  // Four codes a half-word, exact in fp32; 2^23 puts that integer in the low mantissa bits.
  float w[2];
#pragma unroll
  for (int n = 0; n < 2; ++n) w[n] = fmaf(c[4 * n + 3], 4096.f, fmaf(c[4 * n + 2], 256.f, fmaf(c[4 * n + 1], 16.f, c[4 * n]))) + 8388608.f;
  return __byte_perm(__float_as_uint(w[0]), __float_as_uint(w[1]), 0x5410);
}

// The 8 values that a word of codes stands for.
template <typename T>
__device__ __forceinline__ uint4 values8(uint32_t code, uint32_t param) {
  const float s = bits_to_f<T>(param & 0xffffu), z = bits_to_f<T>(param >> 16);
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    w[e] = pack2<T>(fmaf(s, (float)((code >> (8 * e)) & 15u), z), fmaf(s, (float)((code >> (8 * e + 4)) & 15u), z));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int W>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t* r) {
  if constexpr (W == 4) *reinterpret_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
  else if constexpr (W == 2) *reinterpret_cast<uint2*>(p) = make_uint2(r[0], r[1]);
  else {
#pragma unroll
    for (int w = 0; w < W; ++w) reinterpret_cast<uint32_t*>(p)[w] = r[w];
  }
}
template <int W>
__device__ __forceinline__ void load_words(uint32_t* r, const uint8_t* p) {
  if constexpr (W == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
  } else if constexpr (W == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r[0] = v.x; r[1] = v.y;
  } else {
#pragma unroll
    for (int w = 0; w < W; ++w) r[w] = reinterpret_cast<const uint32_t*>(p)[w];
  }
}

// The work of a warp: L rows that end at position len - 1 touch at most tiles_of(L) tiles.
__host__ __device__ __forceinline__ int tiles_of(int L) { return (L + 14) / kTile + 1; }

struct Place {
  int b, h, len, pos0;  // pos0: position of the tile's first row (negative before the start)
  int v, hf;            // 0: keys, 1: values; half of the tile's rows
  bool any;             // whether the warp has work
};
__device__ __forceinline__ Place place_of(const CacheArgs& c, unsigned kid) {
  const int tiles = tiles_of(c.L);
  int64_t w = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  Place p;
  p.any = w < (int64_t)c.B * c.Hkv * tiles * 4;
  if (!p.any) return p;
  p.v = (int)(w & 1);
  p.hf = (int)(w >> 1 & 1);
  w >>= 2;
  const int tile = (int)(w % tiles);
  p.h = (int)(w / tiles % c.Hkv);
  p.b = (int)(w / tiles / c.Hkv);
  p.len = cache_len(c, p.b, c.pages_per_seq * c.page_size, kid);
  p.pos0 = (((p.len - c.L) >> 4) + tile) * kTile;  // >> rounds down
  p.any = p.pos0 < p.len;
  return p;
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) cache_write_kernel(CacheArgs c) {
  using Tl = Tile<D>;
  constexpr int W = Tl::W, JB = Tl::JB;
  const Place p = place_of(c, kKidCacheWrite);
  if (!p.any) return;
  const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int count = c.counts ? min(max(c.counts[p.b], 0), c.L) : c.L;
  const int first = max(0, p.len - count);  // positions first..len-1 are written
  const int v = p.v, hf = p.hf;
  if (p.pos0 + 8 * hf + 8 <= first || p.pos0 + 8 * hf >= p.len) return;
  const int page = cache_page(c, p.b, p.pos0, kKidCacheWrite);
  if (page < 0) return;
  uint8_t* tile = cache_tile<D>(c, page, p.h, p.pos0 % c.page_size / kTile);
  auto written = [&](int r) { return p.pos0 + r >= first && p.pos0 + r < p.len; };
  const int r = g + 8 * hf, i = p.pos0 + r - (p.len - c.L);  // this lane's row, in the tile and of the call
  const T* src = row_ptr<T>(v ? c.v : c.k, v ? c.lv : c.lk, p.b, p.h, i) + 8 * t;
  uint4 in[JB][W];
#pragma unroll
  for (int jb = 0; jb < JB; ++jb)
#pragma unroll
    for (int w = 0; w < W; ++w) {
      in[jb][w] = make_uint4(0, 0, 0, 0);
      if (written(r)) in[jb][w] = *reinterpret_cast<const uint4*>(src + 32 * (jb * W + w));
    }
#pragma unroll
  for (int jb = 0; jb < JB; ++jb) {
    uint32_t code[W], mine = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      uint32_t param;
      code[w] = quantise<T>(in[jb][w], param);
      if (w == t) mine = param;
    }
    uint8_t* words = tile + (v ? Tl::kV : Tl::kK) + ((hf * JB + jb) * 32 + lane) * W * 4;
    if (v == 0) {
      if (written(r)) store_words<W>(words, code);
    } else {
#pragma unroll
      for (int w = 0; w < W; ++w) code[w] = transpose8(code[w]);
      const bool low = written(2 * t + 8 * hf), high = written(2 * t + 1 + 8 * hf);
      if (low && high) {
        store_words<W>(words, code);
      } else if (low || high) {
#pragma unroll
        for (int w = 0; w < W; ++w) reinterpret_cast<uint16_t*>(words)[2 * w + (low ? 0 : 1)] = (uint16_t)(low ? code[w] : code[w] >> 16);
      }
    }
    if (t < W && written(r)) reinterpret_cast<uint32_t*>(tile + (v ? Tl::kVp : Tl::kKp))[(jb * 16 + r) * W + t] = mine;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) cache_read_kernel(CacheArgs c) {
  using Tl = Tile<D>;
  constexpr int W = Tl::W, JB = Tl::JB;
  const Place p = place_of(c, kKidCacheRead);
  if (!p.any) return;
  const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  int page = -1;
  if (p.pos0 >= 0) page = cache_page(c, p.b, p.pos0, kKidCacheRead);
  const uint8_t* tile = page < 0 ? nullptr : cache_tile<D>(c, page, p.h, p.pos0 % c.page_size / kTile);
  const int v = p.v, hf = p.hf, i = p.pos0 + g + 8 * hf - (p.len - c.L);
  uint32_t code[JB][W] = {}, param[JB][W] = {};
  if (tile) {
#pragma unroll
    for (int jb = 0; jb < JB; ++jb) {
      load_words<W>(code[jb], tile + (v ? Tl::kV : Tl::kK) + ((hf * JB + jb) * 32 + lane) * W * 4);
      load_words<W>(param[jb], tile + (v ? Tl::kVp : Tl::kKp) + (jb * 16 + g + 8 * hf) * W * 4);
    }
  }
  T* dst = row_ptr<T>(v ? c.v : c.k, v ? c.lv : c.lk, p.b, p.h, i) + 8 * t;
#pragma unroll
  for (int jb = 0; jb < JB; ++jb)
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint32_t x = v ? transpose8(code[jb][w]) : code[jb][w];
      if (i >= 0 && i < c.L) *reinterpret_cast<uint4*>(dst + 32 * (jb * W + w)) = values8<T>(x, param[jb][w]);
    }
}

template <typename T, int D>
cudaError_t launch_t(const CacheArgs& c, bool write, cudaStream_t s) {
  const unsigned blocks = (unsigned)(((int64_t)c.B * c.Hkv * tiles_of(c.L) * 4 + kWarps - 1) / kWarps);
  if (write) cache_write_kernel<T, D><<<blocks, kWarps * 32, 0, s>>>(c);
  else cache_read_kernel<T, D><<<blocks, kWarps * 32, 0, s>>>(c);
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
