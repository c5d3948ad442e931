// Attention over a 4-bit paged cache (format and conventions in include/sdpa.h).
//
// Rows.  The G·L query rows of a KV head (row r = query r % L of head r / L of the group) are
// cut into row tiles of 4, 8 or 16; a block takes one row tile and one chunk of the sequence, and
// its warps take units of UT tiles (16 tokens each) of that chunk in turn.  Chunks' partial
// results are joined by a second kernel, placed while the first still runs (programmatic
// dependent launch); a sequence of one chunk needs none.
//
// Bound.  5 bits an element from HBM, 1.25·D bytes a token and KV head; everything between
// that and the result is made cheap enough to hide behind it:
//  - A tile is stored in the order in which the lanes of a warp read MMA fragments, so each
//    warp streams its tiles into a shared-memory ring of its own with plain bulk copies (one
//    per tile, issued a few units ahead, no tensor map, no block barrier) and reads fragments
//    with 16-byte loads.
//  - Key codes are not converted.  A nibble masked in place is a subnormal fp16 number, 16·code·2^-24
//    in bits 4 to 7, which the tensor cores multiply exactly; the factors are undone in fp32 scales.
//    (In bits 0 to 3, two shifts a word less, sums keep fewer low bits: at one token scores were
//    off by 8.7e-7 rms in fp16 and 3.3e-7 in bf16, so 0.9e-7 and 0.6e-7.)
//  - The product is transposed, S^T = K·Q^T and O^T = V^T·P^T (m16n8k16), so that the cache is
//    the 16-row operand and 8 query rows fill the other one.
//  - Scales stay outside the products: S = sum_j s_j·(c_j·q_j) + sum_j z_j·sum(q_j) over the
//    groups j, the first in fp32 FMAs over one accumulator a group, the second as one MMA in
//    the element type whose q sums are split in three so that nothing is lost.
//  - For the values the probabilities take the scale: O = sum P·s·(c - 8) + sum P·(z + 8·s), the
//    second in fp32 FMAs.  The 8 costs an fp16 operation for two codes (one sequence 35.6 us
//    without, 39.5 with): an MMA cuts off what falls below the last bit of its sum, and sums of
//    codes of 0 to 15 grow to hundreds of times an output, so that a seventh of the bf16 outputs
//    of 131072 tokens were rounded the other way; now 3 in 10000, fewer than with fp32 matrix
//    products.  (A second MMA that takes 8 off, 37.7 us, leaves 2 in 100.)
//    P·s, times a power of two, enters as two fp16 numbers, its leading 11 bits and what they
//    leave, 2^-21 relative in all and 2^-22 of the largest P·s; the first alone, cheaper by 5 us in
//    the drafts below, would change one output in ten.  So nothing is rounded to fewer bits than
//    fp32 sums show but the output.
//  - fp16 has 40 binades, P·s in bf16 over 250.  So every row has a power of two for each group
//    of values, chosen from products P·s that the row has really seen: a key that it does not
//    see, or whose weight is nothing, does not move it, whatever its values.  They seldom move:
//    a warp looks at P·s only when a score passes the row's reference or a scale of the unit
//    passes what the powers in use allow, a vote a unit.
//
// Measured (bf16, 32 query and 8 KV heads, D = 128, a call replayed from a graph): one sequence of
// 131072 tokens 39.5 us, 168 MB, 4.2 TB/s (kernel alone 37.9 us under ncu with a cold L2, 57% of
// DRAM's peak, issue slots 62%, ALU 59%: bound by its instructions on 12 warps an SM; 31 us with
// the arithmetic of the units left out, of which the first copies' chain of lookups takes some 2.5).
// 32 sequences of 256 to 8192 tokens 49.2 us, 174 MB, 3.5 TB/s.  Eight queries each of 4 sequences of
// 2048 to 8192 (32 rows a KV head, 27 MB) 40.1 us: issue slots 46%, ALU 34%, tensor pipe 24%, so bound
// by the latency of dependent instructions, with two warps a scheduler at 255 registers.
#include <atomic>

#include "cache.h"
#include "tc_common.cuh"

namespace sdpa {
namespace {

// NT: row tiles of 8 rows that a block takes, CW: columns of the transposed products that a
// lane holds.  CW = 2 is the plain form.  CW = 1 is the form for up to 4 rows, which would leave
// half of the 8 columns empty: row r is column 2r, so that every lane has one row and half the
// elements of the softmax and of the scalings.  Its odd columns are zero in the scores; in the
// values they take the remainders of P·s, which need a second MMA in the plain form.
template <int D, int NT, int CW>
struct Cfg {
  using Tl = Tile<D>;
  static constexpr int UT = D <= 64 ? 4 : D <= 128 ? 2 : 1;  // tiles a unit
  static constexpr int kUnit = UT * kTile;                    // tokens a unit
  // Warps a block, and blocks an SM.  The narrow form ran best on 12 warps of up to 168 registers
  // an SM (131072 tokens, D = 128: 39.5 us; 8 warps of 182 registers 42.7; 16 warps of 128
  // registers, which spill, 43.8; 20 of 96, 55.8).
  static constexpr int kWarps = CW == 1 ? 4 : 8;
  static constexpr int kBlocks = CW == 1 ? 3 : NT == 1 && D <= 128 ? 2 : 1;
  static constexpr int kStages = 2;  // a third one: 40.0 us, and one block of the 8-row form instead of two
  static constexpr int kUnitBytes = UT * Tl::kBytes;
  static constexpr int kSlab = 4 * CW;       // rows of a row tile
  static constexpr int kRows = kSlab * NT;
  static constexpr int kRing = kWarps * kStages * kUnitBytes;
  static constexpr int kMerge = kWarps * kSlab * (D + 4) * 4;  // a slab of rows of every warp's output
  static constexpr int kBody = kRing > kMerge ? kRing : kMerge;
  static constexpr int kQ = kBody;                              // q fragments: [group][NT][lane] of 16 bytes
  static constexpr int kSums = kQ + NT * Tl::NG * 32 * 16;      // q's group sums, fp32 [row][group]
  static constexpr int kUnits = kSums + kRows * Tl::NG * 4;     // the scores' units, float2 [row]
  static constexpr int kPowers = kUnits + kRows * 8;            // each warp's powers of two, fp32 [warp][group][row]
  static constexpr int kSmem = kPowers + kWarps * Tl::NG * kRows * 4;
};

using tc::ex2;

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with an accumulator of zero.
template <typename T>
__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// The codes in two of a word's nibbles, less 8, as fp16: the nibble under the exponent of 1024 is
// 1024 + c, or, one place higher, 1024 + 16·c.
__device__ __forceinline__ uint32_t low_codes(uint32_t x) {
  const uint32_t b = (x & 0x000f000fu) | 0x64006400u;
  const __half2 h = __hadd2(*reinterpret_cast<const __half2*>(&b), __float2half2_rn(-1032.f));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t high_codes(uint32_t x) {
  const uint32_t b = (x & 0x00f000f0u) | 0x64006400u;
  const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&b), __float2half2_rn(0.0625f), __float2half2_rn(-72.f));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127 (0 for -127)
__device__ __forceinline__ int exponent(float x) { return (__float_as_int(x) >> 23) - 127; }  // of x >= 0: floor(log2 x), -127 below 2^-126
constexpr int kFree = 119;  // exponent of a power of two that nothing has fixed yet

__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(tc::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}

// Tokens that some row of row tile `rt` (rows a tile) sees: those before this position.
__device__ __forceinline__ int tile_end(const CacheAttnArgs& a, int len, int rt, int rows) {
  if (!a.causal) return len;
  const int R = a.G * a.c.L, r0 = rt * rows, n = min(rows, R - r0), i0 = r0 % a.c.L;
  const int last = i0 + n >= a.c.L ? a.c.L - 1 : i0 + n - 1;  // the latest query among them
  return max(0, len - a.c.L + last + 1);
}

template <typename T, int D, int NT, int CW>
__global__ void __launch_bounds__(Cfg<D, NT, CW>::kWarps * 32, Cfg<D, NT, CW>::kBlocks) cache_attn_kernel(CacheAttnArgs a, int chunk, int splits, int row_tiles) {
  using C = Cfg<D, NT, CW>;
  constexpr int kWarps = C::kWarps;
  using Tl = Tile<D>;
  constexpr int NG = Tl::NG, W = Tl::W, JB = Tl::JB, UT = C::UT;
  constexpr bool kQSmem = NT > 1, kHalf = std::is_same<T, __half>::value;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kWarps][C::kStages];
  __shared__ float stat[kWarps][C::kRows][2];
  __shared__ int abort_flag;
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int split = blockIdx.x, b = blockIdx.z, h = row_tiles == 1 ? blockIdx.y : blockIdx.y / row_tiles, rt = blockIdx.y - h * row_tiles;
  // This warp's query rows, on their way while the length and the pages are looked up.
  const int R = a.G * c.L, row0 = rt * C::kRows;
  constexpr int kMine = (C::kRows + kWarps - 1) / kWarps;
  T q_in[kMine][NG];
#pragma unroll
  for (int n = 0; n < kMine; ++n) {
    const int rr = warp + n * kWarps, r = row0 + rr, head = c.L == 1 ? r : r / c.L;
    const T* q = rr < C::kRows && r < R ? row_ptr<T>(a.q, a.lq, b, h * a.G + head, r - head * c.L) + lane : nullptr;
#pragma unroll
    for (int j = 0; j < NG; ++j) q_in[n][j] = q ? q[32 * j] : Elem<T>::from_f(0.f);
  }
  // Lane st·UT + i looks at tile i of this warp's unit for stage st; the entry is read beside the
  // length, which says whether it counts.
  const int* table = c.pages + b * c.pages_stride;
  const int64_t first = (int64_t)split * chunk;
  int pos = (int)first + (warp + lane / UT * kWarps) * C::kUnit + lane % UT * kTile;
  int slot = (unsigned)pos / (unsigned)c.page_size, off = pos - slot * c.page_size;
  const int entry = lane < C::kStages * UT && slot < c.pages_per_seq ? table[slot] : -1;
  const int len = cache_len(c, b, a.max_len, kKidCacheAttn);
  const int end_all = tile_end(a, len, rt, C::kRows);
  if (first >= end_all && splits > 1) {
    asm volatile("griddepcontrol.launch_dependents;");
    return;
  }
  const int start = (int)first, end = (int)min((int64_t)end_all, first + chunk);
  const int units = end > start ? (end - start + C::kUnit - 1) / C::kUnit : 0;

  // ---- the first copies
  if (lane < C::kStages) {
    tc::mbar_init(&full[warp][lane], 1);
    tc::fence_mbar_init();
  }
  if (threadIdx.x == 0) abort_flag = 0;
  __syncwarp();
  const tc::WaitCtx wc{&abort_flag, 0, a.wait_limit_ns, c.err, kKidCacheAttn};
  uint8_t* ring = smem + warp * (C::kStages * C::kUnitBytes);
  const int64_t page_bytes = (int64_t)c.Hkv * (c.page_size / kTile) * Tl::kBytes;
  const uint8_t* head = c.data + (int64_t)h * (c.page_size / kTile) * Tl::kBytes;
  // The page of a tile at position pos: -1 if the tile is past the end, or the page bad.
  auto checked = [&](int page, int pos) {
    if (pos >= end) return -1;
    if ((unsigned)page < (unsigned)c.num_pages) return page;
    report_error(c.err, kDevErrIndex, kKidCacheAttn);
    return -1;
  };
  // The lanes that looked a page up start with its tile.  Later lane i copies tile i of every unit:
  // it keeps that tile's position, its place in the table and its offset in the page, which move
  // on by a fixed step, and has its page looked up one unit ahead.
  int page = lane < C::kStages * UT ? checked(entry, pos) : -1;
  uint32_t there = __ballot_sync(0xffffffffu, page >= 0);  // bit st·UT + i: tile i of stage st is copied
  if (lane < C::kStages && warp + lane * kWarps < units)
    tc::mbar_arrive_expect_tx(&full[warp][lane], __popc((there >> (lane * UT)) & ((1u << UT) - 1)) * Tl::kBytes);
  __syncwarp();
  if (page >= 0) bulk_copy(ring + lane * Tl::kBytes, head + page * page_bytes + off / kTile * Tl::kBytes, Tl::kBytes, &full[warp][lane / UT]);
  const int step_slots = kWarps * C::kUnit / c.page_size, step_off = kWarps * C::kUnit % c.page_size;
  auto advance = [&] {
    pos += kWarps * C::kUnit;
    slot += step_slots;
    off += step_off;
    if (off >= c.page_size) {
      off -= c.page_size;
      ++slot;
    }
  };
#pragma unroll
  for (int n = 0; n < C::kStages; ++n) advance();
  page = lane < UT && pos < end ? checked(table[slot], pos) : -1;
  // Starts the copies of this warp's next unit into stage s (all lanes call it).
  auto issue = [&](int s) {
    const uint32_t ok = __ballot_sync(0xffffffffu, page >= 0);
    there = (there & ~(((1u << UT) - 1) << (s * UT))) | (ok << (s * UT));
    if (lane == 0) tc::mbar_arrive_expect_tx(&full[warp][s], __popc(ok) * Tl::kBytes);
    __syncwarp();
    if (page >= 0)
      bulk_copy(ring + s * C::kUnitBytes + lane * Tl::kBytes, head + page * page_bytes + off / kTile * Tl::kBytes, Tl::kBytes, &full[warp][s]);
    advance();
    page = lane < UT && pos < end ? checked(table[slot], pos) : -1;
  };
  int issued = warp + C::kStages * kWarps;  // next unit to start

  // ---- query rows as the B operand, through shared memory.  A row is multiplied by the power of
  // two that brings its largest element to 2^13..2^14 (exact in fp16 down to 2^-27 of that), and by
  // the sign of the scale, so that the largest score is the largest accumulator (0 for a scale of
  // zero).  Lane (g, t) of a fragment has row g's elements 8t..8t+7 of a group.
  uint16_t* const q_frag = reinterpret_cast<uint16_t*>(smem + C::kQ);
  float* const q_sum = reinterpret_cast<float*>(smem + C::kSums);
  // A score is its accumulator times |scale|·log2e·2^(kUp - e), one fp32 number f unless that is
  // far from 1 (a row of large elements; a scale of 1e30): then f is about its square root, and
  // accumulators are multiplied by the other root first, a power of two.
  constexpr int kUp = 20;
  float2* const q_unit = reinterpret_cast<float2*>(smem + C::kUnits);
  bool far = false;
#pragma unroll
  for (int n_row = 0; n_row < kMine; ++n_row) {
    const int rr = warp + n_row * kWarps;
    if (rr >= C::kRows) break;
    float x[NG], top = 0.f;
#pragma unroll
    for (int j = 0; j < NG; ++j) x[j] = Elem<T>::to_f(q_in[n_row][j]);
#pragma unroll
    for (int j = 0; j < NG; ++j) top = fmaxf(top, fabsf(x[j]));
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    // A row of zeros (or subnormals) takes 2^126; one with an infinity 2^-115, and turns NaN by itself.
    const int e = min(126, 13 - ((__float_as_int(top) >> 23) - 127));
    const float up = a.scale_mant == 0.f ? 0.f : copysignf(pow2(e), a.scale_mant);
    const int nt = CW == 2 ? rr / 8 : 0, g_row = CW == 2 ? rr % 8 : 2 * rr;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      x[j] *= up;
      const int n = lane % 8;  // element 8·(lane / 8) + n of the group
      q_frag[((j * NT + nt) * 32 + g_row * 4 + lane / 8) * 8 + n % 4 * 2 + n / 4] = (uint16_t)f_to_bits<__half>(x[j]);
    }
#pragma unroll
    for (int j = 0; j < NG; ++j) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) x[j] += __shfl_xor_sync(0xffffffffu, x[j], off);
      if (lane == j) q_sum[rr * NG + j] = x[j];
    }
    const int u = a.scale_exp + kUp - e, root = u / 2;
    const bool wide = a.scale_mant != 0.f && (u < -100 || u > 100);
    far = far || wide;
    if (lane == 0) {
      const float mant = a.scale_mant == 0.f ? 1.f : fabsf(a.scale_mant);
      if (wide) q_unit[rr] = make_float2(mant * pow2(max(-126, min(127, u - root))), pow2(max(-126, min(127, root))));
      else q_unit[rr] = make_float2(a.scale_mant == 0.f ? 1.f : mant * pow2(u), 1.f);
    }
  }
  far = __syncthreads_or(far);
  // The z term's share has bf16's range to be in the accumulators' units (2^-20: the codes are 16
  // times theirs) at once; in fp16 it stays at 2^13 or less and is scaled after its MMA.
  constexpr float kZUp = kHalf ? 0x1p-6f : 0x1p-20f;
  const uint4* qs = reinterpret_cast<const uint4*>(smem + C::kQ);
  const bool row_here = CW == 2 || g % 2 == 0;  // odd columns of the narrow form are zero
  uint32_t qf[kQSmem ? 1 : NG][4];
  if constexpr (!kQSmem) {
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row_here) v = qs[j * 32 + lane];
      qf[j][0] = v.x; qf[j][1] = v.y; qf[j][2] = v.z; qf[j][3] = v.w;
    }
  }
  uint32_t qz[NT][JB][2];  // group sums of the row, split in three (z term)
  float f[NT][CW];         // per row of this lane's columns: score per accumulator, > 0
  int lim[NT][CW];         // the same: positions below this are visible
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int jb = 0; jb < JB; ++jb) {  // sums·kZUp = hi + mid + lo in T
      float sum = 0.f;
      if (row_here && (W == 4 || t < W)) sum = q_sum[(CW == 2 ? 8 * nt + g : g / 2) * NG + 4 * jb + t] * kZUp;
      const uint32_t hi = f_to_bits<T>(sum);
      const float rest = sum - bits_to_f<T>(hi);
      const uint32_t mid = f_to_bits<T>(rest);
      qz[nt][jb][0] = hi | (mid << 16);
      qz[nt][jb][1] = f_to_bits<T>(rest - bits_to_f<T>(mid));
    }
#pragma unroll
    for (int n = 0; n < CW; ++n) {  // the accumulators' columns are 2t and 2t + 1
      const int rr = C::kSlab * nt + CW * t + n;
      f[nt][n] = q_unit[rr].x;
      lim[nt][n] = a.causal ? len - c.L + (row0 + rr) % c.L + 1 : len;
    }
  }
  const int seen = a.causal ? len - c.L + 1 : len;  // every row sees the positions below this

  float o[2 * NG][NT][4];  // wt·sum of P·s·(c - 8)
  float zo[NT][NG][CW];    // this lane's keys' P·(z + 8·s)
  float m[NT][CW], l[NT][CW];  // reference (P <= 1), sum
  float wt[NT][NG][CW];    // P·s enters the MMA times this power of two, at most 2^15
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < 2 * NG; ++j) o[j][nt][0] = o[j][nt][1] = o[j][nt][2] = o[j][nt][3] = 0.f;
#pragma unroll
    for (int n = 0; n < CW; ++n) {
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        zo[nt][j][n] = 0.f;
        wt[nt][j][n] = pow2(kFree);
      }
      m[nt][n] = minus_inf();
      l[nt][n] = 0.f;
    }
  }
  uint32_t slimit[JB];  // scales of group 4·jb + t whose bits reach this call for other powers
#pragma unroll
  for (int jb = 0; jb < JB; ++jb) slimit[jb] = 1;
  float* const powers = reinterpret_cast<float*>(smem + C::kPowers) + warp * (NG * C::kRows);
  bool fresh = true;  // no unit yet

  // One unit in shared memory: scores, softmax, values.  Only units that a sequence's or a
  // row's end cuts, or that lack a tile, take the masked form.
  auto unit = [&](const uint8_t* st, int key0, uint32_t tiles, auto masked) {
    constexpr bool kMasked = decltype(masked)::value;
    // All ones where key g + 8·hf of tile ti is there, and where this lane's row sees it.  What
    // differs from lane to lane is arithmetic on such words, not a branch: the MMAs and transposes
    // need the whole warp at once, and a compiler may copy what follows a branch into its arms.
    auto key_there = [&](int ti, int hf) { return (uint32_t)((key0 + ti * kTile + g + 8 * hf - end) >> 31) & (0u - ((tiles >> ti) & 1)); };
    auto seen_by = [&](int ti, int hf, int nt, int n) { return (uint32_t)((key0 + ti * kTile + g + 8 * hf - lim[nt][n]) >> 31); };
    const int tw = W == 4 ? t : min(t, W - 1);  // lanes beyond the groups repeat the last one
    // ---- scores
    float sc[UT][NT][2][CW];  // [.][.][half][n]: key g + 8·half, this lane's column n
#pragma unroll
    for (int ti = 0; ti < UT; ++ti) {
      const uint8_t* tile = st + ti * Tl::kBytes;
      float acc[NT][4];
#pragma unroll
      for (int jb = 0; jb < JB; ++jb) {  // z of group 4·jb + t: (hi, mid) and (lo, nothing)
        const uint32_t* zp = reinterpret_cast<const uint32_t*>(tile + Tl::kKp) + (jb * 16 + g) * W + tw;
        const uint32_t group_here = W == 4 ? ~0u : (uint32_t)((t - W) >> 31);
        const uint32_t z0 = zp[0] >> 16 & group_here, z1 = zp[8 * W] >> 16 & group_here;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (jb == 0) mma0<T>(acc[nt], z0 * 0x10001u, z1 * 0x10001u, z0, z1, qz[nt][jb][0], qz[nt][jb][1]);
          else mma<T>(acc[nt], z0 * 0x10001u, z1 * 0x10001u, z0, z1, qz[nt][jb][0], qz[nt][jb][1]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int n = 0; n < CW; ++n) sc[ti][nt][hf][n] = kHalf ? acc[nt][2 * hf + n] * 0x1p-14f : acc[nt][2 * hf + n];
    }
#pragma unroll
    for (int jb = 0; jb < JB; ++jb) {
      uint32_t kw[UT][2][W], kp[UT][2][W];
#pragma unroll
      for (int ti = 0; ti < UT; ++ti)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint8_t* tile = st + ti * Tl::kBytes;
          load_words<W>(kw[ti][hf], tile + Tl::kK + ((hf * JB + jb) * 32 + lane) * W * 4);
          load_words<W>(kp[ti][hf], tile + Tl::kKp + (jb * 16 + g + 8 * hf) * W * 4);
        }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const int j = jb * W + w;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t qq[4];
          if constexpr (kQSmem) {
            const uint4 v = qs[(j * NT + nt) * 32 + lane];
            qq[0] = v.x; qq[1] = v.y; qq[2] = v.z; qq[3] = v.w;
          } else {
            qq[0] = qf[j][0]; qq[1] = qf[j][1]; qq[2] = qf[j][2]; qq[3] = qf[j][3];
          }
#pragma unroll
          for (int ti = 0; ti < UT; ++ti) {
            const uint32_t x0 = kw[ti][0][w], x1 = kw[ti][1][w], y0 = x0 >> 8, y1 = x1 >> 8;
            float acc[4];
            mma0<__half>(acc, x0 << 4 & 0x00f000f0u, x1 << 4 & 0x00f000f0u, x0 & 0x00f000f0u, x1 & 0x00f000f0u, qq[0], qq[1]);
            mma<__half>(acc, x0 >> 4 & 0x00f000f0u, x1 >> 4 & 0x00f000f0u, y0 & 0x00f000f0u, y1 & 0x00f000f0u, qq[2], qq[3]);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const float s = bits_to_f<T>(kp[ti][hf][w] & 0xffffu);
#pragma unroll
              for (int n = 0; n < CW; ++n) sc[ti][nt][hf][n] = fmaf(s, acc[2 * hf + n], sc[ti][nt][hf][n]);
            }
          }
        }
      }
    }

    if (far) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int n = 0; n < CW; ++n) {
          const float root = q_unit[C::kSlab * nt + CW * t + n].y;
#pragma unroll
          for (int ti = 0; ti < UT; ++ti) {
            sc[ti][nt][0][n] *= root;
            sc[ti][nt][1][n] *= root;
          }
        }
    }

    // ---- softmax.  The reference m of a row starts 2^8 above its largest score and stays until
    // some score passes it; wt stays until a scale could take P·s·wt over 2^15.  One vote covers
    // both.
    bool move = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int n = 0; n < CW; ++n) {
        float top = minus_inf();
#pragma unroll
        for (int ti = 0; ti < UT; ++ti)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float& x = sc[ti][nt][hf][n];
            if constexpr (kMasked) {
              const uint32_t here = key_there(ti, hf) & seen_by(ti, hf, nt, n);
              x = __uint_as_float((__float_as_uint(x) & here) | (0xff800000u & ~here));
            }
            top = fmaxf(top, x);
          }
        move = move || fmaf(top, f[nt][n], -m[nt][n]) > 0.f;
      }
    uint32_t smax[JB];  // lane (g, t) looks at group 4·jb + t of rows g and g + 8
#pragma unroll
    for (int jb = 0; jb < JB; ++jb) {
      smax[jb] = 0;
#pragma unroll
      for (int ti = 0; ti < UT; ++ti)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t w = reinterpret_cast<const uint32_t*>(st + ti * Tl::kBytes + Tl::kVp)[(jb * 16 + g + 8 * hf) * W + tw];
          if constexpr (kMasked) w &= key_there(ti, hf);
          smax[jb] = __vmaxu2(smax[jb], w);
        }
      smax[jb] &= 0xffffu;  // scales are not negative: their bits order them
      move = move || smax[jb] >= slimit[jb];
    }
    if (__any_sync(0xffffffffu, move)) {
      float al[NT][CW];
      bool plain = fresh;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int n = 0; n < CW; ++n) {
          float top = minus_inf();
#pragma unroll
          for (int ti = 0; ti < UT; ++ti) top = fmaxf(top, fmaxf(sc[ti][nt][0][n], sc[ti][nt][1][n]));
#pragma unroll
          for (int off = 4; off <= 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
          const float m_old = m[nt][n], m_new = fmaf(top, f[nt][n], -m_old) > 0.f ? __fmaf_ru(top, f[nt][n], 8.f) : m_old;
          al[nt][n] = m_new == m_old ? 1.f : ex2(m_old - m_new);
          m[nt][n] = m_new;
          plain = plain && fabsf(m_new) < 0x1p20f;
        }
      // Largest scale (high half) and the complement of the smallest one of group 4·jb + t.
      uint32_t range[JB];
#pragma unroll
      for (int jb = 0; jb < JB; ++jb) {
        range[jb] = 0;
#pragma unroll
        for (int ti = 0; ti < UT; ++ti)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(st + ti * Tl::kBytes + Tl::kVp)[(jb * 16 + g + 8 * hf) * W + tw];
            uint32_t both = w << 16 | (~w & 0xffffu);
            if constexpr (kMasked) both &= key_there(ti, hf);
            range[jb] = __vmaxu2(range[jb], both);
          }
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) range[jb] = __vmaxu2(range[jb], __shfl_xor_sync(0xffffffffu, range[jb], off));
        plain = plain && exponent(bits_to_f<T>(range[jb] >> 16)) - exponent(bits_to_f<T>(~range[jb] & 0xffffu)) <= 4;
      }
      if (__all_sync(0xffffffffu, plain)) {
        // A first unit of the usual kind: every row sees a key, so that its largest P is 2^-8 (less
        // where scores are so large that m is rounded), and no scale is under 2^-5 of its group's
        // largest.  The power that takes that one to 2^10..2^11 then has a product P·s of at least
        // 2^-3 in every row.
        int now[JB];
#pragma unroll
        for (int jb = 0; jb < JB; ++jb) {
          now[jb] = min(kFree - 1, 10 - exponent(bits_to_f<T>(range[jb] >> 16)));
          slimit[jb] = max(1u, f_to_bits<T>(pow2(min(127, 15 - now[jb]))));
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          const float power = pow2(__shfl_sync(0xffffffffu, now[j / W], j % W));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int n = 0; n < CW; ++n) wt[nt][j][n] = power;
        }
      } else {
        // The products themselves, row by row and group by group, in loops that are not unrolled
        // (code that seldom runs costs what it takes to fetch it), with the powers in shared memory.
        float* const mine = powers + CW * t;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int n = 0; n < CW; ++n)
#pragma unroll
            for (int j = 0; j < NG; ++j) mine[j * C::kRows + C::kSlab * nt + n] = wt[nt][j][n];
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int n = 0; n < CW; ++n) {
            const int e_al = al[nt][n] > 0.f ? exponent(al[nt][n]) : -512;  // -512: what was seen before counts for nothing
            float p[UT][2];
#pragma unroll
            for (int ti = 0; ti < UT; ++ti)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) p[ti][hf] = ex2(fmaf(sc[ti][nt][hf][n], f[nt][n], -fmaxf(m[nt][n], -3.4e38f)));
            float* at = mine + C::kSlab * nt + n;
#pragma unroll 1
            for (int j = 0; j < NG; ++j, at += C::kRows) {
              const int jb = JB == 1 ? 0 : j / W, w = JB == 1 ? j : j % W;
              float ps = 0.f;  // the unit's largest P·s (fmaxf drops what is NaN: places without a key)
#pragma unroll
              for (int ti = 0; ti < UT; ++ti)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                  ps = fmaxf(ps, p[ti][hf] * bits_to_f<T>(reinterpret_cast<const uint32_t*>(st + ti * Tl::kBytes + Tl::kVp)[(jb * 16 + g + 8 * hf) * W + w] & 0xffffu));
#pragma unroll
              for (int off = 4; off <= 16; off <<= 1) ps = fmaxf(ps, __shfl_xor_sync(0xffffffffu, ps, off));
              // What the row had seen before was at least 2^-3 / its power.  The new power leaves
              // the largest product so far at 2^-3 or more; above that it is the old one, or the
              // one that takes the unit's largest scale to 2^10..2^11 (P <= 1).
              const int e_s = exponent(bits_to_f<T>(__shfl_sync(0xffffffffu, JB == 1 || j < W ? range[0] : range[JB - 1], w) >> 16));
              const int was = exponent(*at), e_ps = max(exponent(ps), was == kFree ? -127 : e_al - 3 - was);
              __syncwarp();
              *at = pow2(e_ps <= -127 ? kFree : min(kFree - 1, max(-3 - e_ps, min(was, 10 - e_s))));  // (the same in the lanes of a column)
            }
          }
        __syncwarp();
#pragma unroll
        for (int jb = 0; jb < JB; ++jb) {
          float most = 0.f;
#pragma unroll 1
          for (int r = 0; r < C::kRows; ++r) most = fmaxf(most, powers[(jb * W + tw) * C::kRows + r]);
          slimit[jb] = max(1u, f_to_bits<T>(pow2(min(127, 15 - exponent(most)))));
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int n = 0; n < CW; ++n) {
            l[nt][n] *= al[nt][n];
#pragma unroll
            for (int j = 0; j < NG; ++j) {
              const float power = mine[j * C::kRows + C::kSlab * nt + n];
              const float both = al[nt][n] * pow2(max(-127, min(126, exponent(power) - exponent(wt[nt][j][n]))));
              wt[nt][j][n] = power;
              zo[nt][j][n] *= al[nt][n];
#pragma unroll
              for (int jj = 2 * j; jj < 2 * j + 2; ++jj) {
                o[jj][nt][n] *= both;
                o[jj][nt][2 + n] *= both;
                if constexpr (CW == 1) {
                  o[jj][nt][1] *= both;
                  o[jj][nt][3] *= both;
                }
              }
            }
          }
      }
    }
    fresh = false;
    __syncwarp();
#pragma unroll
    for (int ti = 0; ti < UT; ++ti) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int n = 0; n < CW; ++n) {
            const float ref = kMasked ? fmaxf(m[nt][n], -3.4e38f) : m[nt][n];  // -inf while nothing was seen: P = 0
            const float p = ex2(fmaf(sc[ti][nt][hf][n], f[nt][n], -ref));
            sc[ti][nt][hf][n] = p;
            l[nt][n] += p;
          }
      // ---- values
#pragma unroll
      for (int jb = 0; jb < JB; ++jb) {
        uint32_t vw[2][W], vp[2][W];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          load_words<W>(vw[hf], st + ti * Tl::kBytes + Tl::kV + ((hf * JB + jb) * 32 + lane) * W * 4);
          load_words<W>(vp[hf], st + ti * Tl::kBytes + Tl::kVp + (jb * 16 + g + 8 * hf) * W * 4);
          if constexpr (kMasked) {
#pragma unroll
            for (int w = 0; w < W; ++w) vp[hf][w] &= key_there(ti, hf);
          }
        }
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const int j = jb * W + w;
          const uint32_t x0 = vw[0][w], x1 = vw[1][w], y0 = x0 >> 8, y1 = x1 >> 8;
          const uint32_t a0 = low_codes(x0), a1 = high_codes(x0), a2 = low_codes(x1), a3 = high_codes(x1);
          const uint32_t c0 = low_codes(y0), c1 = high_codes(y0), c2 = low_codes(y1), c3 = high_codes(y1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float top[2][CW], rest[2][CW];  // P·s: its leading 11 bits, and the rest
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const float s = bits_to_f<T>(vp[hf][w] & 0xffffu), z = fmaf(8.f, s, bits_to_f<T>(vp[hf][w] >> 16));
#pragma unroll
              for (int n = 0; n < CW; ++n) {
                const float p = sc[ti][nt][hf][n], q = p * wt[nt][j][n] * s;
                top[hf][n] = __uint_as_float(__float_as_uint(q) & 0xffffe000u);
                rest[hf][n] = q - top[hf][n];
                // A hidden key's z may be NaN and counts as 0; a visible one's is seen, whatever its weight.
                if constexpr (kMasked) zo[nt][j][n] = fmaf(p, __uint_as_float(__float_as_uint(z) & seen_by(ti, hf, nt, n)), zo[nt][j][n]);
                else zo[nt][j][n] = fmaf(p, z, zo[nt][j][n]);
              }
            }
            const uint32_t b0 = transpose8(pack2<__half>(top[0][0], CW == 1 ? rest[0][0] : top[0][CW - 1]));
            const uint32_t b1 = transpose8(pack2<__half>(top[1][0], CW == 1 ? rest[1][0] : top[1][CW - 1]));
            mma<__half>(o[2 * j][nt], a0, a1, a2, a3, b0, b1);
            mma<__half>(o[2 * j + 1][nt], c0, c1, c2, c3, b0, b1);
            if constexpr (CW == 2) {
              const uint32_t r0 = transpose8(pack2<__half>(rest[0][0], rest[0][CW - 1]));
              const uint32_t r1 = transpose8(pack2<__half>(rest[1][0], rest[1][CW - 1]));
              mma<__half>(o[2 * j][nt], a0, a1, a2, a3, r0, r1);
              mma<__half>(o[2 * j + 1][nt], c0, c1, c2, c3, r0, r1);
            }
          }
        }
      }
    }
  };

  bool ok = true;
  int s = 0;
  uint32_t parity = 0;
  for (int u = warp; u < units; u += kWarps) {
    ok = __all_sync(0xffffffffu, tc::mbar_wait(&full[warp][s], parity, wc));
    if (!ok) break;
    const uint8_t* st = ring + s * C::kUnitBytes;
    const int key0 = start + u * C::kUnit;
    const uint32_t tiles = (there >> (s * UT)) & ((1u << UT) - 1);
    if (key0 + C::kUnit > min(seen, end) || tiles != (1u << UT) - 1) unit(st, key0, tiles, std::true_type());
    else unit(st, key0, tiles, std::false_type());
    __syncwarp();  // the stage has been read
    if (issued < units) issue(s);
    issued += kWarps;
    if (++s == C::kStages) {
      s = 0;
      parity ^= 1;
    }
  }
  if (!ok) {  // a wait ran out: let this warp's copies in flight end, for as long again
    const uint64_t t0 = tc::globaltimer();
    for (int n = s; n < s + C::kStages; ++n)
      while (!tc::mbar_try_wait(&full[warp][n % C::kStages], parity ^ (n >= C::kStages ? 1u : 0u)) &&
             tc::globaltimer() - t0 < a.wait_limit_ns) {
      }
  }
  if (__syncthreads_or(!ok)) return;  // also: every warp is done with its ring

  // ---- join the warps: statistics, then 8 rows at a time through shared memory
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int n = 0; n < CW; ++n) {
#pragma unroll
      for (int off = 4; off <= 16; off <<= 1) l[nt][n] += __shfl_xor_sync(0xffffffffu, l[nt][n], off);
#pragma unroll
      for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) zo[nt][j][n] += __shfl_xor_sync(0xffffffffu, zo[nt][j][n], off);
      if (g == 0) {
        stat[warp][C::kSlab * nt + CW * t + n][0] = m[nt][n];
        stat[warp][C::kSlab * nt + CW * t + n][1] = l[nt][n];
      }
    }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;");
  float* red = reinterpret_cast<float*>(smem);  // [warp][kSlab][D + 4]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float wgt[CW];
#pragma unroll
    for (int n = 0; n < CW; ++n) {
      float M = minus_inf();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, stat[w][C::kSlab * nt + CW * t + n][0]);
      wgt[n] = m[nt][n] == minus_inf() ? 0.f : ex2(m[nt][n] - M);
    }
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
      for (int n = 0; n < CW; ++n) {
        const float z = zo[nt][j][n];
        const float back = pow2(-exponent(wt[nt][j][n]));
        auto sum = [&](int jj, int hf) { return CW == 1 ? o[jj][nt][2 * hf] + o[jj][nt][2 * hf + 1] : o[jj][nt][2 * hf + n]; };
        float4 v;
        v.x = fmaf(sum(2 * j, 0), back, z) * wgt[n];
        v.y = fmaf(sum(2 * j, 1), back, z) * wgt[n];
        v.z = fmaf(sum(2 * j + 1, 0), back, z) * wgt[n];
        v.w = fmaf(sum(2 * j + 1, 1), back, z) * wgt[n];
        *reinterpret_cast<float4*>(red + (warp * C::kSlab + CW * t + n) * (D + 4) + 32 * j + 4 * g) = v;
      }
    __syncthreads();
    for (int x = threadIdx.x; x < C::kSlab * (D / 4); x += kWarps * 32) {
      const int q = x / (D / 4), d = x % (D / 4) * 4, r = row0 + C::kSlab * nt + q;
      if (r < R) {
        float M = minus_inf(), Lsum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, stat[w][C::kSlab * nt + q][0]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          // A warp without a maximum has seen nothing, or nothing but NaN: its sum is 0 or NaN.
          const float mw = stat[w][C::kSlab * nt + q][0], lw = stat[w][C::kSlab * nt + q][1];
          Lsum += mw == minus_inf() ? lw : lw * ex2(mw - M);
          const float4 y = *reinterpret_cast<const float4*>(red + (w * C::kSlab + q) * (D + 4) + d);
          v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
        }
        const int hq = h * a.G + r / c.L, i = r % c.L;
        const int64_t row = ((int64_t)b * a.Hq + hq) * c.L + i;
        if (splits > 1) {
          const int64_t at = row * splits + split;
          *reinterpret_cast<float4*>(a.workspace + at * D + d) = v;
          if (d == 0) {
            float* ml = a.workspace + (int64_t)c.B * a.Hq * c.L * splits * D + 2 * at;
            ml[0] = M;
            ml[1] = Lsum;
          }
        } else {
          const float fold = fold_sink(a.sinks, hq, M, Lsum), inv = Lsum == 0.f ? 0.f : fold / Lsum;
          T* out = row_ptr<T>(a.out, a.lo, b, hq, i) + d;
          *reinterpret_cast<uint2*>(out) = make_uint2(pack2<T>(v.x * inv, v.y * inv), pack2<T>(v.z * inv, v.w * inv));
          if (a.lse && d == 0) a.lse[row] = Lsum == 0.f ? minus_inf() : (M + log2f(Lsum)) * kLn2;
        }
      }
    }
    __syncthreads();
  }
}

// Joins the chunks of one query row: D/4 threads a chunk, several chunks side by side.
template <typename T, int D, int kJoinThreads>
__global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(CacheAttnArgs a, int chunk, int splits, int rows_a_tile) {
  constexpr int U = D / 4, kSide = kJoinThreads / U;
  __shared__ float4 part[kSide][U];
  __shared__ float red[kJoinThreads / 32], sums[kJoinThreads / 32];
  const CacheArgs& c = a.c;
  const int64_t row = blockIdx.x;
  const int i = (int)(row % c.L), hq = (int)(row / c.L % a.Hq), b = (int)(row / c.L / a.Hq);
  const int len = cache_len(c, b, a.max_len, kKidCacheAttn);
  const int end = tile_end(a, len, (hq % a.G * c.L + i) / rows_a_tile, rows_a_tile);
  const int n = (int)(((int64_t)end + chunk - 1) / chunk);  // chunks that have been written
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float* ml = a.workspace + (int64_t)c.B * a.Hq * c.L * splits * D + 2 * row * splits;
  float M = minus_inf(), L = 0.f;
  for (int x = threadIdx.x; x < n; x += kJoinThreads) M = fmaxf(M, ml[2 * x]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) M = fmaxf(M, red[w]);
  for (int x = threadIdx.x; x < n; x += kJoinThreads)
    L += ml[2 * x] == minus_inf() ? ml[2 * x + 1] : ml[2 * x + 1] * ex2(ml[2 * x] - M);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
  if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = L;
  const int side = threadIdx.x / U, d = threadIdx.x % U * 4;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (side < kSide) {
#pragma unroll 4
    for (int x = side; x < n; x += kSide) {
      const float mx = ml[2 * x], w = mx == minus_inf() ? 0.f : ex2(mx - M);
      const float4 y = *reinterpret_cast<const float4*>(a.workspace + (row * splits + x) * D + d);
      v.x = fmaf(w, y.x, v.x);
      v.y = fmaf(w, y.y, v.y);
      v.z = fmaf(w, y.z, v.z);
      v.w = fmaf(w, y.w, v.w);
    }
    part[side][d / 4] = v;
  }
  __syncthreads();
  if (threadIdx.x >= U) return;
  L = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) L += sums[w];
  v = part[0][d / 4];
  for (int x = 1; x < kSide; ++x) {
    const float4 y = part[x][d / 4];
    v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
  }
  const float fold = fold_sink(a.sinks, hq, M, L), inv = L == 0.f ? 0.f : fold / L;
  T* out = row_ptr<T>(a.out, a.lo, b, hq, i) + d;
  *reinterpret_cast<uint2*>(out) = make_uint2(pack2<T>(v.x * inv, v.y * inv), pack2<T>(v.z * inv, v.w * inv));
  if (a.lse && d == 0) a.lse[row] = L == 0.f ? minus_inf() : (M + log2f(L)) * kLn2;
}

// How a call is cut.
struct Plan {
  int cw, nt, row_tiles, chunk, splits, rows;
};

Plan make_plan(const CacheAttnArgs& a) {
  Plan p;
  const int R = a.G * a.c.L;
  // The forms, both sides of each border measured (131072 tokens, 4 rows): plain 51.9 us, narrow
  // 39.6; 8192 tokens, 32 rows: tiles of 8 rows 44.1 us, of 16 40.1, of 32 (which spill) 60.9.
  p.cw = R <= 4 ? 1 : 2;
  p.nt = R <= 8 ? 1 : 2;
  p.rows = 4 * p.cw * p.nt;
  p.row_tiles = (R + p.rows - 1) / p.rows;
  const int step = 256;  // tokens: a unit or two a warp
  const int64_t slots = (int64_t)(a.c.num_sms > 0 ? a.c.num_sms : 1) * (p.cw == 1 ? 3 : p.nt == 1 && a.c.D <= 128 ? 2 : 1);
  const int64_t pairs = (int64_t)a.c.B * a.c.Hkv * p.row_tiles;
  // Few pairs: one wave of blocks, whatever the chunk.  Many: chunks short enough that sequences of
  // unequal length share the SMs (32 of 256..8192 tokens: 2048 tokens 53.4 us, 1536 49.2, 1024 49.0,
  // 512 52.5; 32 rows: 47.9, 40.1, 43.2, 48.3).  Equal shares of all tokens, cut on the device, ran
  // slower (with the units at 41.9 and 33.8 us: 49.5, and 36.9 for one sequence): finding a share
  // costs 1.7 us, each further sequence in it about 4.
  const int64_t want = max((int64_t)1, slots / pairs);
  int64_t chunk = (a.max_len + want - 1) / want;
  if (pairs * 4 > slots) chunk = min(chunk, (int64_t)1536);
  // A second chunk costs the join, some 1.5 us, whatever it saves: none while one block's warps read
  // the sequence in less.  One call of 8 KV heads, whole against chunks of 256: D = 128, 512 tokens,
  // 6.5 us, 7.1, 1024 tokens 10.1, 7.1; D = 64, 1024 tokens 6.9, 6.5; D = 256, 512 tokens 13.0, 10.1;
  // 32 rows (D = 64) 512 tokens 7.6, 8.7, 1024 tokens 10.2, 9.1.  Longer ones: chunks of at least
  // 256 (1024 to 4096 tokens, D = 128: 7.1 to 8.0 us; of 512 8.8 to 9.3, of 128 6.8 to 7.8, but 10.0
  // instead of 9.4 for 32 rows of 1024).
  const int whole = min(1024, (p.nt == 1 ? 65536 : 32768) / a.c.D);
  chunk = a.max_len <= whole ? a.max_len : max(chunk, (int64_t)step);
  // Partial results take at most 64 MiB, half of L2: beyond that there are more than 2000 blocks of
  // 16 rows (8000 of 4) anyway, and a workspace that grew with the table would reach gigabytes.
  const int64_t partial = (int64_t)a.c.B * a.Hq * a.c.L * (a.c.D + 2) * (int64_t)sizeof(float);
  const int64_t most = max((int64_t)1, ((int64_t)64 << 20) / partial);
  chunk = max(chunk, (a.max_len + most - 1) / most);
  p.chunk = (int)min((chunk + step - 1) / step * step, (int64_t)1 << 30);
  p.splits = (a.max_len + p.chunk - 1) / p.chunk;
  return p;
}

template <typename T, int D, int NT, int CW>
cudaError_t attn_nt(const CacheAttnArgs& a, const Plan& p, cudaStream_t s) {
  using C = Cfg<D, NT, CW>;
  auto* kern = cache_attn_kernel<T, D, NT, CW>;
  // The shared-memory limit is set once on each device.
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  kern<<<dim3(p.splits, p.row_tiles * a.c.Hkv, a.c.B), C::kWarps * 32, C::kSmem, s>>>(a, p.chunk, p.splits, p.row_tiles);
  return cudaGetLastError();
}

template <typename T, int D, int kThreads>
cudaError_t join_t(const CacheAttnArgs& a, const Plan& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.c.B * a.Hq * a.c.L));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];  // its blocks may be placed while the last chunks are still running
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_join_kernel<T, D, kThreads>, a, p.chunk, p.splits, p.rows);
}

template <typename T, int D>
cudaError_t attn_t(const CacheAttnArgs& a, bool join, cudaStream_t s) {
  const Plan p = make_plan(a);
  if (!join) {
    if (p.cw == 1) return attn_nt<T, D, 1, 1>(a, p, s);
    switch (p.nt) {
      case 1: return attn_nt<T, D, 1, 2>(a, p, s);
      default: return attn_nt<T, D, 2, 2>(a, p, s);
    }
  }
  // A row of few chunks is joined by four warps; with many, 16 warps read them side by side
  // (131072 tokens in 57 chunks: 42.0 us a call with 4 warps, 39.6 with 16; 6 chunks: 49.2, 54.7).
  return p.splits > 16 ? join_t<T, D, 512>(a, p, s) : join_t<T, D, 128>(a, p, s);
}

template <typename T>
cudaError_t attn_d(const CacheAttnArgs& a, bool join, cudaStream_t s) {
  switch (a.c.D) {
    case 32: return attn_t<T, 32>(a, join, s);
    case 64: return attn_t<T, 64>(a, join, s);
    case 96: return attn_t<T, 96>(a, join, s);
    case 128: return attn_t<T, 128>(a, join, s);
    case 256: return attn_t<T, 256>(a, join, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t attn_any(const CacheAttnArgs& a, int dtype, bool join, cudaStream_t s) {
  if (dtype == 1) return attn_d<__half>(a, join, s);
  if (dtype == 2) return attn_d<__nv_bfloat16>(a, join, s);
  return cudaErrorInvalidValue;
}

}  // namespace

size_t cache_attn_workspace(const CacheAttnArgs& a) {
  const Plan p = make_plan(a);
  return p.splits == 1 ? 0 : (size_t)a.c.B * a.Hq * a.c.L * p.splits * (a.c.D + 2) * sizeof(float);
}

int cache_attn_row_tiles(const CacheAttnArgs& a) { return make_plan(a).row_tiles; }

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int dtype, cudaStream_t s) { return attn_any(a, dtype, false, s); }
cudaError_t launch_cache_join(const CacheAttnArgs& a, int dtype, cudaStream_t s) { return attn_any(a, dtype, true, s); }

}  // namespace sdpa
