// Rotary embedding of q and k by positions on one or several axes, and its inverse (which
// is also its gradient): one kernel, one launch for both tensors.
//
// Pair p of a row turns by the angle position·inv_freq[p].  Far positions make that angle
// thousands of turns, of which only the fraction counts, so it is computed modulo one turn in
// 64-bit integers: inv_freq/2π as a fraction of 2^64 (a 24-bit mantissa times 2^64/2π,
// shifted), times the position, wraps by itself.  No fp64 and no range reduction is left: the
// top two bits are the quadrant, the rest is an angle within π/4 of it.
//
// Bound: HBM (each element read and written once).  A block takes a few tokens: its threads
// compute their sines and cosines once, into shared memory, while the first heads' loads are
// on their way; then a thread keeps those of VP pairs of one token in registers and turns that
// token's heads hg, hg + HG, ... in 16-byte pieces.
// Measured (bf16, B = 2, 32 + 8 heads, L = 4096, D = 128; 168 MB): 31.3 us a call from a graph,
// 5.4 TB/s, 0.79 of the copy rate; waiting on loads (long scoreboard 8.8 of 14 cycles a warp and
// instruction).  With the sines computed by every thread for 8 heads (64-bit divisions, CUDA's
// sincospif) it took 35 to 50 us; fp32 (B = 8, 8 + 8 heads, L = 577, D = 64) 7.5 us, 5.0 TB/s.
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

// Cosine and sine of a phase in units of 2^-64 turns.  x in [-π/4, π/4] is the distance from
// the nearest quarter turn, 3·2^-24 of itself off (two roundings and the constant's), so that
// small sines and cosines keep their digits (from the phase's upper 32 bits alone the sine of 2e-6
// would be 7e-4 of itself off; the wider conversion costs nothing that shows).  Taylor's series to
// x^9 and x^10 leave 2e-9 and 5e-10; with their last roundings both are within 5·2^-24 of themselves.
__device__ __forceinline__ float2 cos_sin(uint64_t phase) {
  const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
  const float x = (float)(int64_t)(phase - ((uint64_t)quarter << 62)) * 3.4061215800687046e-19f;  // 2π / 2^64
  const float y = x * x;
  const float s = fmaf(x * y, fmaf(y, fmaf(y, fmaf(y, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), x);
  const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
  const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
  return make_float2(((quarter + 1) & 2) ? -a : a, (quarter & 2) ? -b : b);
}

template <typename T, int N>
struct __align__(N * sizeof(T)) Vec {
  T v[N];
};

__device__ __forceinline__ void turn(float& u, float& w, float c, float s) {
  const float a = u * c - w * s;
  w = w * c + u * s;
  u = a;
}

// Turns VP pairs: x[e], y[e], or (adjacent) x[2e], x[2e + 1].  16-bit elements are unpacked and
// packed two at a time.
template <typename T, bool ADJ, int VP>
__device__ __forceinline__ void turn_pairs(Vec<T, ADJ ? 2 * VP : VP>& x, Vec<T, ADJ ? 2 * VP : VP>& y, const float (&cs)[VP], const float (&sn)[VP]) {
  if constexpr (sizeof(T) == 2 && (ADJ || VP % 2 == 0)) {
    uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
    uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
    for (int e = 0; e < (ADJ ? VP : VP / 2); ++e) {
      float a = bits_to_f<T>(xw[e] & 0xffffu), b = bits_to_f<T>(xw[e] >> 16);
      if constexpr (ADJ) {
        turn(a, b, cs[e], sn[e]);
      } else {
        float c = bits_to_f<T>(yw[e] & 0xffffu), d = bits_to_f<T>(yw[e] >> 16);
        turn(a, c, cs[2 * e], sn[2 * e]);
        turn(b, d, cs[2 * e + 1], sn[2 * e + 1]);
        yw[e] = pack2<T>(c, d);
      }
      xw[e] = pack2<T>(a, b);
    }
  } else {
#pragma unroll
    for (int e = 0; e < VP; ++e) {
      T& u = ADJ ? x.v[2 * e] : x.v[e];
      T& w = ADJ ? x.v[2 * e + 1] : y.v[e];
      float a = Elem<T>::to_f(u), b = Elem<T>::to_f(w);
      turn(a, b, cs[e], sn[e]);
      u = Elem<T>::from_f(a);
      w = Elem<T>::from_f(b);
    }
  }
}

// VP pairs a thread: vectors of VP elements at p and p + rot/2, or one of 2·VP adjacent ones.
// VP = 1 is the form for any rot.
template <typename T, bool ADJ, int VP>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(RotaryArgs a, int slots, int tail, int tokens, int groups) {
  constexpr int NV = ADJ ? 2 * VP : VP;  // elements a vector
  // Heads of a batch; the next batch is loaded while one is turned.  16-bit types 1 (62.0 us for
  // two calls; 2, which needs 80 registers, 73.7; without the batch ahead 2 took 63.2), fp32 2
  // (15.0 us; 1: 15.7; 4 without the batch ahead 16.8).
  constexpr int kBatch = sizeof(T) == 4 ? 2 : 1;
  using V = Vec<T, NV>;
  extern __shared__ __align__(16) float tables[];  // cosines, then sines: [tokens][rot / 2]
  const int half = a.rot / 2, all = slots + tail, H = a.Hq + a.Hkv;
  const unsigned row0 = blockIdx.x * tokens, rows = (unsigned)a.B * a.L;  // fewer than 2^31
  const int slot = threadIdx.x % all, token = threadIdx.x / all % tokens, group = threadIdx.x / all / tokens;
  const unsigned row = row0 + token;
  const bool here = group < groups && row < rows;
  const int b = here ? row / (unsigned)a.L : 0, i = here ? row - b * a.L : 0;
  // Row i of batch b: where its first head is, for each of the four tensors.
  const T* q = row_ptr<T>(a.q, a.lq, b, 0, i);
  const T* k = row_ptr<T>(a.k, a.lk, b, 0, i);
  T* q_out = row_ptr<T>(a.q_out, a.lqo, b, 0, i);
  T* k_out = row_ptr<T>(a.k_out, a.lko, b, 0, i);
  const int at0 = slot < slots ? slot * NV : a.rot + (slot - slots) * NV;  // this thread's elements
  const int step = gridDim.y * groups;
  V x[2][kBatch], y[2][kBatch];
  auto load = [&](int hb, V (&x)[kBatch], V (&y)[kBatch]) {  // heads hb, hb + step, ...: their loads are in flight together
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const int h = hb + n * step;
      if (h >= H) continue;
      const T* src = (h < a.Hq ? q + h * a.lq.sh : k + (h - a.Hq) * a.lk.sh) + at0;
      x[n] = *reinterpret_cast<const V*>(src);
      if (!ADJ && slot < slots) y[n] = *reinterpret_cast<const V*>(src + half);
    }
  };
  const int first = blockIdx.y * groups + group;
  if (here) load(first, x[0], y[0]);
  const int pair = threadIdx.x % half, stride = kThreads / half;  // a pair, and every stride-th token
  if (threadIdx.x < stride * half) {
    int axis = a.axes ? a.axes[pair] : 0;
    if ((unsigned)axis >= (unsigned)a.naxes) {
      report_error(a.err, kDevErrIndex, kKidRotary);
      axis = 0;
    }
    const float f = a.inv_freq[pair];
    const uint64_t step_phase = turns_per_step(f);
    for (int tk = threadIdx.x / half; tk < tokens && row0 + tk < rows; tk += stride) {
      const unsigned r = row0 + tk, rb = r / (unsigned)a.L;
      const int64_t at = axis * a.pos_axis + rb * a.pos_batch + (r - rb * a.L) * a.pos_row;
      const int64_t pos = a.pos64 ? static_cast<const int64_t*>(a.positions)[at] : static_cast<const int32_t*>(a.positions)[at];
      float2 cs = cos_sin(step_phase * (uint64_t)pos);
      if (!isfinite(f)) cs.x = cs.y = __int_as_float(0x7fffffff);
      tables[tk * half + pair] = cs.x;
      tables[(tokens + tk) * half + pair] = a.inverse ? -cs.y : cs.y;
    }
  }
  __syncthreads();
  if (!here) return;
  float cs[VP], sn[VP];
#pragma unroll
  for (int e = 0; e < VP; ++e) {
    const int p = token * half + (slot < slots ? slot * VP : 0) + e;
    cs[e] = tables[p];
    sn[e] = tables[tokens * half + p];
  }
  auto finish = [&](int hb, V (&x)[kBatch], V (&y)[kBatch]) {
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const int h = hb + n * step;
      if (h >= H) continue;
      T* dst = (h < a.Hq ? q_out + h * a.lqo.sh : k_out + (h - a.Hq) * a.lko.sh) + at0;
      if (slot >= slots) {  // elements past rot are copied
        *reinterpret_cast<V*>(dst) = x[n];
        continue;
      }
      turn_pairs<T, ADJ, VP>(x[n], y[n], cs, sn);
      *reinterpret_cast<V*>(dst) = x[n];
      if (!ADJ) *reinterpret_cast<V*>(dst + half) = y[n];
    }
  };
  const int ahead = kBatch * step;
  for (int hb = first; hb < H; hb += 2 * ahead) {
    if (hb + ahead < H) load(hb + ahead, x[1], y[1]);
    finish(hb, x[0], y[0]);
    if (hb + 2 * ahead < H) load(hb + 2 * ahead, x[0], y[0]);
    if (hb + ahead < H) finish(hb + ahead, x[1], y[1]);
  }
}

template <typename T, bool ADJ, int VP>
cudaError_t rotary_t(const RotaryArgs& a, cudaStream_t s) {
  constexpr int NV = ADJ ? 2 * VP : VP;
  const int slots = a.rot / 2 / VP, tail = (a.D - a.rot) / NV, all = slots + tail, H = a.Hq + a.Hkv;
  const int64_t rows = (int64_t)a.B * a.L, sms = a.num_sms > 0 ? a.num_sms : 1;
  // Up to 32 tokens a block, fewer while that leaves less than 3 blocks an SM (1: 80.9 us for two
  // calls, 2 or 3: 63.3, 8: 66.6); the threads that are left split the heads, and blocks split them
  // too if there are still few.
  int tokens = max(1, min(32, kThreads / all));
  while (tokens > 1 && (rows + tokens - 1) / tokens < 3 * sms) tokens /= 2;
  const int groups = max(1, min(H, kThreads / (all * tokens)));
  const int64_t blocks = (rows + tokens - 1) / tokens;
  const int splits = (int)max((int64_t)1, min((int64_t)((H + groups - 1) / groups), 2 * sms / blocks));
  rotary_kernel<T, ADJ, VP><<<dim3((unsigned)blocks, splits), kThreads, tokens * a.rot * sizeof(float), s>>>(a, slots, tail, tokens, groups);
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
