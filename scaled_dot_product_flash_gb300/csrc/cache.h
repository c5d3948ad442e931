// Internal parameters and launchers of the rotary embedding and of the 4-bit paged cache,
// and the layout of a cache tile (documented in include/sdpa.h).
#pragma once

#include "common.cuh"

namespace sdpa {

struct RotaryArgs {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const void* positions;  // [naxes, B, L], int32 or int64
  bool pos64;
  int64_t pos_axis, pos_batch, pos_row;  // element strides
  const float* inv_freq;                 // [rot / 2]
  const int* axes;                       // [rot / 2], or null: axis 0
  int naxes, B, Hq, Hkv, L, D, rot;      // Hkv = 0 without k
  bool adjacent, inverse;
  Layout lq, lk, lqo, lko;
  unsigned* err;
  int num_sms;
};
cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t s);

// A cache and one call's page table and lengths.
struct CacheArgs {
  uint8_t* data;
  int num_pages, page_size, Hkv, D;
  const int* pages;
  int64_t pages_stride;
  int pages_per_seq;
  const int* lens;
  int B, L;  // L: rows of the call (queries, for attention)
  unsigned* err;
  int num_sms;
  // write: inputs; read: outputs
  void* k;
  void* v;
  Layout lk, lv;
  const int* counts;
};
cudaError_t launch_cache_write(const CacheArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_cache_read(const CacheArgs& a, int dtype, cudaStream_t s);

struct CacheAttnArgs {
  CacheArgs c;
  const void* q;
  void* out;
  float* lse;          // nullable
  const float* sinks;  // nullable
  Layout lq, lo;
  int Hq, G;
  float scale_mant;    // scale·log2e = scale_mant·2^scale_exp, |scale_mant| in [1/2, 1) or 0
  int scale_exp;
  int causal;
  int max_len;         // longest sequence, in tokens
  float* workspace;
  uint64_t wait_limit_ns;
};
size_t cache_attn_workspace(const CacheAttnArgs& a);  // 0: one kernel does it all
int cache_attn_row_tiles(const CacheAttnArgs& a);
cudaError_t launch_cache_attn(const CacheAttnArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_cache_join(const CacheAttnArgs& a, int dtype, cudaStream_t s);  // after it, with a workspace

constexpr int kTile = 16;   // tokens a tile
constexpr int kGroup = 32;  // elements that share a scale and a zero

// Offsets inside a tile of 20·D bytes.
template <int D>
struct Tile {
  static constexpr int NG = D / kGroup;
  static constexpr int W = NG < 4 ? NG : 4;
  static constexpr int JB = NG / W;
  static constexpr int kK = 0, kV = 8 * D, kKp = 16 * D, kVp = 18 * D, kBytes = 20 * D;
  // Lane 4g + t of a warp reads the K and V codes as pieces [row half][jb][lane] of W words, and
  // the parameters of row r as piece [jb][r] of W words (s in the low half, z in the high one).
};

// Tokens of sequence b that a call may touch: lens[b] within 0..most, reported otherwise.
__device__ __forceinline__ int cache_len(const CacheArgs& c, int b, int most, unsigned kid) {
  const int n = c.lens[b];
  if (n < 0 || n > most) report_error(c.err, kDevErrIndex, kid);
  return n < 0 ? 0 : (n > most ? most : n);
}

// Page of position `pos` (0 <= pos < pages_per_seq·page_size) of sequence b, or -1, reported.
__device__ __forceinline__ int cache_page(const CacheArgs& c, int b, int pos, unsigned kid) {
  const int page = c.pages[b * c.pages_stride + pos / c.page_size];
  if ((unsigned)page < (unsigned)c.num_pages) return page;
  report_error(c.err, kDevErrIndex, kid);
  return -1;
}

template <int D>
__device__ __forceinline__ uint8_t* cache_tile(const CacheArgs& c, int page, int h, int tile) {
  return c.data + (((int64_t)page * c.Hkv + h) * (c.page_size / kTile) + tile) * Tile<D>::kBytes;
}

// 16-bit element bits <-> fp32.
template <typename T>
__device__ __forceinline__ float bits_to_f(uint32_t x);
template <>
__device__ __forceinline__ float bits_to_f<__half>(uint32_t x) { return __half2float(__ushort_as_half((unsigned short)x)); }
template <>
__device__ __forceinline__ float bits_to_f<__nv_bfloat16>(uint32_t x) { return __uint_as_float(x << 16); }
template <typename T>
__device__ __forceinline__ uint32_t f_to_bits(float x);
template <>
__device__ __forceinline__ uint32_t f_to_bits<__half>(float x) { return __half_as_ushort(__float2half_rn(x)); }
template <>
__device__ __forceinline__ uint32_t f_to_bits<__nv_bfloat16>(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

// Two values rounded to 16-bit elements, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Transposes an 8 x 8 matrix of 16-bit elements held two a lane, by the whole warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// W 32-bit words of a tile.
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

}  // namespace sdpa
