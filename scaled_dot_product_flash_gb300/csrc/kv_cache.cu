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
// reverse), launch latency for single tokens.  Measured (bf16, 8 heads, D = 128): two prompts of
// 4096 tokens written in 15.7 us under ncu, 44 MB, 2.8 TB/s: a warp loads its half tile, waits and
// then has some 19 instructions an element and lane (issue slots 70%, ALU 52%, warps active 52%, no
// load ahead of the arithmetic); the last 8192 rows of four prefixes of 2048 to 8192 read back in
// 26.7 us from a graph, 160 MB, 6.0 TB/s, 0.88 of the copy rate.  A thread an 8-element piece with 2-byte stores of the value halves took 31 us and
// 41 us.  Half a tile of keys or of values a warp: a whole tile a warp was as fast on prompts, but
// one token's write and read took 15.2 us instead of 7.3, on one warp's chain of 16 groups.
#include "cache.h"

namespace sdpa {
namespace {

constexpr int kWarps = 8;

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

// Minimum and maximum that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Quotients rounded correctly from a reciprocal rounded correctly, one residual step (Markstein
// 1990): a few instructions instead of a division's, for values whose residual does not underflow.
__device__ __forceinline__ float quotient(float a, float d, float inv) {
  const float q = __fmul_rn(a, inv);
  return fmaf(fmaf(-q, d, a), inv, q);
}

// Codes, scale and zero of a group of 32 elements held by the 4 lanes of a quad, 8 each.
// Returns this lane's 8 codes (nibble n = x[n]) and the parameter word (s | z << 16).
template <typename T>
__device__ __forceinline__ uint32_t quantise(const uint4& in, uint32_t& param) {
  constexpr float kInf = __builtin_huge_valf();
  // Scales from here on are normal numbers of T, so that no quotient exceeds 15.5, and far from
  // fp32's smallest.  Others take the form below that divides and clamps.
  constexpr float kPlain = std::is_same<T, __half>::value ? 0x1p-14f : 0x1p-100f;
  float x[8];
  unpack8<T>(x, in);
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    lo = min_nan(lo, x[e]);
    hi = max_nan(hi, x[e]);
  }
#pragma unroll
  for (int off = 1; off <= 2; off <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
  }
  const float range = __fsub_rn(hi, lo);
  if (!(range < kInf)) {  // an element that is not finite, or too wide a range
    param = f_to_bits<T>(__int_as_float(0x7fffffff)) << 16;
    return 0;
  }
  const uint32_t sb = f_to_bits<T>(range > 0x1p-100f ? quotient(range, 15.f, 1.f / 15.f) : __fdiv_rn(range, 15.f));
  param = sb | (f_to_bits<T>(lo) << 16);
  const float s = bits_to_f<T>(sb);
  float c[8];
  if (s >= kPlain) {
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = quotient(__fsub_rn(x[e], lo), s, inv);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = s > 0.f ? fminf(__fdiv_rn(__fsub_rn(x[e], lo), s), 15.f) : 0.f;
  }
  // Adding 1.5·2^23 rounds to an integer, ties to even, in the low mantissa bits; the bits above
  // them are the same eight times over and leave with one constant, modulo 2^32.
  constexpr uint32_t kMagic = 0x4b400000u;
  uint32_t word = 0u - kMagic * 0x11111111u;
#pragma unroll
  for (int e = 0; e < 8; ++e) word += __float_as_uint(__fadd_rn(c[e], 12582912.f)) * (1u << (4 * e));
  return word;
}

// The 8 values that a word of codes stands for.  A nibble under the exponent of 1024 is
// 1024 + code in fp16 (1024 + 16·code, one nibble higher), two of them a word.
template <typename T>
__device__ __forceinline__ uint4 values8(uint32_t code, uint32_t param) {
  const float s = bits_to_f<T>(param & 0xffffu), z = bits_to_f<T>(param >> 16), s16 = s * 0.0625f;
  float x[8];
#pragma unroll
  for (int n = 0; n < 4; ++n) {  // nibbles n and n + 4
    const uint32_t w = n < 2 ? code : code >> 8;
    const uint32_t bits = n % 2 ? (w & 0x00f000f0u) | 0x64006400u : (w & 0x000f000fu) | 0x64006400u;
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&bits), __half2half2(__float2half_rn(1024.f)));
    x[n] = fmaf(n % 2 ? s16 : s, __low2float(h), z);
    x[n + 4] = fmaf(n % 2 ? s16 : s, __high2float(h), z);
  }
  return make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
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

// The work of a warp: L rows that end at position len - 1 touch at most tiles_of(L) tiles.
__host__ __device__ __forceinline__ int tiles_of(int L) { return (L + 14) / kTile + 1; }

struct Place {
  int b, h, len, pos0;  // pos0: position of the tile's first row (negative before the start)
  int v, hf;            // 0: keys, 1: values; half of the tile's rows
  bool any;             // whether the warp has work
};
// The grid is (tiles, heads, sequences).
__device__ __forceinline__ Place place_of(const CacheArgs& c, unsigned kid) {
  const int w = blockIdx.x * kWarps + threadIdx.x / 32;
  Place p;
  p.b = blockIdx.z;
  p.h = blockIdx.y;
  p.v = w & 1;
  p.hf = w >> 1 & 1;
  p.any = w >> 2 < tiles_of(c.L);
  if (!p.any) return p;
  p.len = cache_len(c, p.b, c.pages_per_seq * c.page_size, kid);
  p.pos0 = (((p.len - c.L) >> 4) + (w >> 2)) * kTile;  // >> rounds down
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
  // Past the table's end no new row has a place: the tokens that are there stay.
  const int len = c.lens[p.b], room = c.pages_per_seq * c.page_size;
  if (len > room && len - count >= room) return;
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
      __syncwarp();  // the transposes need the whole warp, whose lanes' groups took different branches
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
  if (v) {  // before the stores, which only some lanes make
    __syncwarp();
#pragma unroll
    for (int jb = 0; jb < JB; ++jb)
#pragma unroll
      for (int w = 0; w < W; ++w) code[jb][w] = transpose8(code[jb][w]);
  }
  __syncwarp();
  if (i < 0 || i >= c.L) return;
#pragma unroll
  for (int jb = 0; jb < JB; ++jb)
#pragma unroll
    for (int w = 0; w < W; ++w) *reinterpret_cast<uint4*>(dst + 32 * (jb * W + w)) = values8<T>(code[jb][w], param[jb][w]);
}

template <typename T, int D>
cudaError_t launch_t(const CacheArgs& c, bool write, cudaStream_t s) {
  const dim3 blocks((unsigned)((tiles_of(c.L) * 4u + kWarps - 1) / kWarps), c.Hkv, c.B);
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
