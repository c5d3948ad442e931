// Rotary embedding of q and k by positions on one or several axes, and its inverse (which
// is also its gradient): one kernel, one launch for both tensors.
//
// Pair p of a row turns by the angle position·inv_freq[p].  Far positions make that angle
// thousands of turns, of which only the fraction counts, so it is computed modulo one turn in
// 64-bit integers: inv_freq/2π as a fraction of 2^64 (a 24-bit mantissa times 2^64/2π,
// shifted), times the position, wraps by itself.  No fp64 and no range reduction is left;
// sincospif takes the signed top 32 bits.
//
// Bound: HBM (each element read and written once; a sine and a cosine a pair and token,
// shared by the heads).  A thread keeps the sines and cosines of VP pairs of one token in
// registers and runs over a range of heads with 16-byte loads and stores.
#include "cache.h"

namespace sdpa {
namespace {

constexpr int kThreads = 256;

// f/2π modulo 1 in units of 2^-64, truncated: the phase of one position step.
__device__ __forceinline__ uint64_t turns_per_step(float f) {
  constexpr uint64_t k2p64Over2Pi = 0x28BE60DB9391054Aull;  // floor(2^64 / 2π)
  const uint32_t bits = __float_as_uint(f);
  const int e = (bits >> 23) & 0xff;
  const uint64_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  const uint64_t lo = m * k2p64Over2Pi, hi = __umul64hi(m, k2p64Over2Pi);
  const int sh = (e ? e : 1) - 150;  // f = m·2^sh
  uint64_t r;
  if (sh >= 0) r = sh < 64 ? lo << sh : 0;
  else if (sh > -64) r = (hi << (64 + sh)) | (lo >> -sh);
  else r = sh > -128 ? hi >> (-sh - 64) : 0;
  return (bits >> 31) ? 0 - r : r;
}

template <typename T, int N>
struct __align__(N * sizeof(T)) Vec {
  T v[N];
};

// VP pairs a thread: PAIRED vectors of VP elements at p and p + rot/2, or one of 2·VP
// adjacent ones.  VP = 1 is the form for any rot.
template <typename T, bool ADJ, int VP>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs a, int slots, int tail, int rows_per_block, int heads) {
  constexpr int NV = ADJ ? 2 * VP : VP;  // elements a vector
  using V = Vec<T, NV>;
  const int all = slots + tail;
  const int lrow = threadIdx.x / all, slot = threadIdx.x % all;
  const int64_t row = (int64_t)blockIdx.x * rows_per_block + lrow;
  if (lrow >= rows_per_block || row >= (int64_t)a.B * a.L) return;
  const int b = (int)(row / a.L), i = (int)(row % a.L);
  const int h0 = blockIdx.y * heads, h1 = min(h0 + heads, a.Hq + a.Hkv);
  if (slot >= slots) {  // elements past rot are copied
    const int d = a.rot + (slot - slots) * NV;
    for (int h = h0; h < h1; ++h) {
      const bool is_q = h < a.Hq;
      const T* src = is_q ? row_ptr<T>(a.q, a.lq, b, h, i) : row_ptr<T>(a.k, a.lk, b, h - a.Hq, i);
      T* dst = is_q ? row_ptr<T>(a.q_out, a.lqo, b, h, i) : row_ptr<T>(a.k_out, a.lko, b, h - a.Hq, i);
      if (dst != src) *reinterpret_cast<V*>(dst + d) = *reinterpret_cast<const V*>(src + d);
    }
    return;
  }
  const int p0 = slot * VP, half = a.rot / 2;
  float cs[VP], sn[VP];
#pragma unroll
  for (int e = 0; e < VP; ++e) {
    int axis = a.axes ? a.axes[p0 + e] : 0;
    if ((unsigned)axis >= (unsigned)a.naxes) {
      report_error(a.err, kDevErrIndex, kKidRotary);
      axis = 0;
    }
    const int64_t at = axis * a.pos_axis + b * a.pos_batch + i * a.pos_row;
    const int64_t pos = a.pos64 ? static_cast<const int64_t*>(a.positions)[at] : static_cast<const int32_t*>(a.positions)[at];
    const float f = a.inv_freq[p0 + e];
    const uint64_t phase = turns_per_step(f) * (uint64_t)pos;
    const float x = (float)(int32_t)(uint32_t)(phase >> 32) * 0x1p-31f;  // half turns in [-1, 1]
    sincospif(x, &sn[e], &cs[e]);
    if (!isfinite(f)) cs[e] = sn[e] = __int_as_float(0x7fffffff);
    if (a.inverse) sn[e] = -sn[e];
  }
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const bool is_q = h < a.Hq;
    const T* src = is_q ? row_ptr<T>(a.q, a.lq, b, h, i) : row_ptr<T>(a.k, a.lk, b, h - a.Hq, i);
    T* dst = is_q ? row_ptr<T>(a.q_out, a.lqo, b, h, i) : row_ptr<T>(a.k_out, a.lko, b, h - a.Hq, i);
    if (ADJ) {
      V x = *reinterpret_cast<const V*>(src + 2 * p0);
#pragma unroll
      for (int e = 0; e < VP; ++e) {
        const float u = Elem<T>::to_f(x.v[2 * e]), w = Elem<T>::to_f(x.v[2 * e + 1]);
        x.v[2 * e] = Elem<T>::from_f(u * cs[e] - w * sn[e]);
        x.v[2 * e + 1] = Elem<T>::from_f(w * cs[e] + u * sn[e]);
      }
      *reinterpret_cast<V*>(dst + 2 * p0) = x;
    } else {
      V x = *reinterpret_cast<const V*>(src + p0), y = *reinterpret_cast<const V*>(src + p0 + half);
#pragma unroll
      for (int e = 0; e < VP; ++e) {
        const float u = Elem<T>::to_f(x.v[e]), w = Elem<T>::to_f(y.v[e]);
        x.v[e] = Elem<T>::from_f(u * cs[e] - w * sn[e]);
        y.v[e] = Elem<T>::from_f(w * cs[e] + u * sn[e]);
      }
      *reinterpret_cast<V*>(dst + p0) = x;
      *reinterpret_cast<V*>(dst + p0 + half) = y;
    }
  }
}

template <typename T, bool ADJ, int VP>
cudaError_t rotary_t(const RotaryArgs& a, cudaStream_t s) {
  constexpr int NV = ADJ ? 2 * VP : VP;
  const int slots = a.rot / 2 / VP, tail = (a.D - a.rot) / NV;
  const int rows = kThreads / (slots + tail);
  const int64_t blocks = ((int64_t)a.B * a.L + rows - 1) / rows;
  const int H = a.Hq + a.Hkv;
  // Heads are split over blocks until there are some 8 blocks an SM.
  const int64_t want = 8 * (int64_t)(a.num_sms > 0 ? a.num_sms : 1);
  const int splits = (int)min((int64_t)H, max((int64_t)1, (want + blocks - 1) / blocks));
  const int heads = (H + splits - 1) / splits;
  rotary_kernel<T, ADJ, VP><<<dim3((unsigned)blocks, (H + heads - 1) / heads), kThreads, 0, s>>>(a, slots, tail, rows, heads);
  return cudaGetLastError();
}

template <typename T>
cudaError_t rotary_any(const RotaryArgs& a, cudaStream_t s) {
  constexpr int kVec = 16 / (int)sizeof(T);  // elements of a 16-byte vector
  if (a.adjacent) {
    if (a.rot % kVec == 0) return rotary_t<T, true, kVec / 2>(a, s);
    return rotary_t<T, true, 1>(a, s);
  }
  if (a.rot / 2 % kVec == 0) return rotary_t<T, false, kVec>(a, s);
  return rotary_t<T, false, 1>(a, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t s) {
  switch (dtype) {
    case 0: return rotary_any<float>(a, s);
    case 1: return rotary_any<__half>(a, s);
    case 2: return rotary_any<__nv_bfloat16>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
