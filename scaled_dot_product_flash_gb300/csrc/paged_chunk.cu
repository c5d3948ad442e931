// Attention over a 16-bit paged cache for many query rows a KV head: TMA + tcgen05 + TMEM
// (conventions in include/sdpa.h).
//
// Rows.  A Q tile of 128 rows holds `tokens` consecutive queries of `heads` query heads of one KV
// head (row = token·heads + head), the split of the group's heads that needs the fewest tiles, so
// that short chunks fill a tile with the heads that share its keys, and the rows of a tile end at
// almost the same token under the causal mask.  One box of the tensor map of q loads them, the same
// box of the map of out stores them; rows that the split leaves over are zeros.
// Keys.  A tile of 128 keys is put together from the pages: boxes of as many tokens as page size
// and tile have in common (16 to 128), one lane each, at the place that the page table names; boxes
// past the last key, or on a bad page, are loaded from outside the tensor, which fills zeros.  Values
// behind the sequence's last token are cleared in shared memory before they meet P.
//
// The pipeline is that of the dense forward kernel: a block of 12 warps computes two Q tiles;
// warps 0-3 / 4-7 are the softmax of tile 0 / 1, one thread a row; warp 8 loads; warps 9 / 10
// issue the MMAs of tile 0 / 1; warp 11 looks whether all pages are good.  S_w = Q_w·K^T goes to TMEM
// columns [128w, 128w + 128), P_w over its first 64 as the A operand of O_w += P_w·V at columns
// [256 + 128w, +D), PV in two halves of 64 keys.  The two softmax warpgroups take turns at the
// exponentials.  The base of a row's exponents follows its scores lazily (paged.h).  Rows that see few keys
// take P as head and remainder (16 more bits), see split_tile.  What does not fill a wave of blocks is cut
// along the keys, and the join kernel adds the unnormalised results up.
//
// Bound: the tensor pipe, 1024 cycles a pair of tiles of 128 x 128 at D = 128; exponentials take half of that.
// Measured (bf16, 32 query and 8 KV heads, D = 128, from a graph): 2 prompts of 4096 tokens 230 us, 1195
// TFLOP/s, 0.62 of the measured rate (the dense kernel on the same shape 228); 2048 queries over 32768
// tokens 765 us, 1400 TFLOP/s, 0.73; in fp16 236 to 240 and 780 to 800.  A block's iteration takes some 3000
// cycles for 2048 of the tensor pipe, its start and end some 5 us.  The softmax loop is sensitive: clearing V's
// last rows in it, once a block, cost 3%, looking values of cut tiles through 5 to 9%, rounding c·s before
// the base is taken off it 4%.
#include "paged_tc.cuh"

namespace sdpa {
namespace {
using namespace tc;

constexpr int kStages = 4;      // ring of K and V tiles
constexpr int kThreads = 384;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kScanWarp = 11;
// The block is launched with 168 registers a thread: 128·56 + 256·224 = 384·168.
constexpr int kRegsLow = 56, kRegsHigh = 224;

template <int D>
struct Layout128 {
  static constexpr int kCB = (D + 63) / 64;  // blocks of 64 elements
  static constexpr int kTileBytes = kBM * kCB * 128;
  static constexpr int kQOff = 0, kRingOff = 2 * kTileBytes;
  static constexpr int kBytes = kRingOff + kStages * kTileBytes + 1024;
};

struct Bars {
  uint64_t q_full, kv_full[kStages], kv_empty[kStages];
  uint64_t s_full[2], p_half[2], p_full[2], o_done[2], mma_done[2], turn[2], scanned, tail_clean;
  uint32_t tmem_base;
  int abort, bad_pages;
};

// What a block of Q tiles works on.
struct Work {
  int b, h, group, i0;  // sequence, KV head, group of its query heads, first query
  int split, k_lo;      // chunk of keys
  bool cut;             // it is one of several
};
__device__ __forceinline__ Work work_of(const PagedArgs& a, const Tiling& t, int queries) {
  // All sequences and heads of the last block of queries, then of the one before: under the causal
  // mask the heaviest first, so that the tail of the grid is light.
  const int units = a.c.B * a.c.Hkv * t.groups;
  const int unit = blockIdx.x % units, rank = blockIdx.x / units;
  Work w;
  w.group = unit % t.groups;
  w.h = unit / t.groups % a.c.Hkv;
  w.b = unit / t.groups / a.c.Hkv;
  w.cut = rank >= t.whole;
  const int block = w.cut ? t.whole + (rank - t.whole) / t.cut.splits : rank;
  w.split = w.cut ? (rank - t.whole) % t.cut.splits : 0;
  w.i0 = (t.blocks - 1 - block) * queries;
  w.k_lo = (int)min((int64_t)w.split * t.cut.chunk, (int64_t)1 << 30);
  return w;
}

// One Q tile: its queries [i0, i1), the keys that some row of it sees in this chunk, and those
// that every real row sees.
struct Span {
  int i0, i1, end, least;
};
__device__ __forceinline__ Span span_of(const Rows& rows, const Tiling& t, int i0, const Work& w) {
  Span s;
  s.i0 = i0;
  s.i1 = min(rows.L, i0 + t.tokens);
  const bool any = i0 < s.i1 && s.i1 > rows.first;
  s.end = any ? (w.cut ? (int)min((int64_t)rows.limit(s.i1 - 1), (int64_t)w.k_lo + t.cut.chunk) : rows.limit(s.i1 - 1)) : 0;
  s.least = any ? rows.limit(max(i0, rows.first)) : 0;
  return s;
}
__device__ __forceinline__ int tiles_in(const Span& s, int k_lo) { return s.end > k_lo ? (s.end - k_lo + kBN - 1) / kBN : 0; }

// A KV tile takes P as head and remainder where some row may see few keys: |O| can then lie near
// the largest values, and P's rounding would add to O as much as O's own.
__device__ __forceinline__ bool split_tile(const Span& s, int k0) { return k0 == 0 && s.least <= kBN; }

// Whether a page table entry that the keys [lo, hi) need is bad (a warp).
__device__ __forceinline__ bool pages_bad(const CacheArgs& c, const int* table, int lo, int hi) {
  bool bad = false;
  if (hi > lo) {
    const int last = (hi - 1) / c.page_size;
    for (int e0 = lo / c.page_size + threadIdx.x % 32; e0 <= last; e0 += 256) {  // eight on their way at once
      int page[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) page[x] = e0 + 32 * x <= last ? table[e0 + 32 * x] : 0;
#pragma unroll
      for (int x = 0; x < 8; ++x) bad |= (unsigned)page[x] >= (unsigned)c.num_pages;
    }
  }
  if (bad) report_error(c.err, kDevErrIndex, kKidPagedAttn);
  return __any_sync(0xffffffffu, bad);
}

// Hides the keys of bad pages in a row of scores; returns the factor that the scores then take.
__device__ __forceinline__ float hide_bad_pages(uint32_t (&sv)[kBN], const CacheArgs& c, const int* table, int k0, int end, float scale2) {
  const int lane = threadIdx.x % 32, pos = k0 + lane * kTile;
  const bool fine = lane >= kBN / kTile || pos >= end || (unsigned)table[pos / c.page_size] < (unsigned)c.num_pages;
  const uint32_t ok = __ballot_sync(0xffffffffu, fine);
  // (a scale of zero would turn the hidden ones into NaN)
#pragma unroll
  for (int e = 0; e < kBN; ++e) {
    if (scale2 == 0.f) sv[e] = 0u;
    if (!(ok >> (e / kTile) & 1u)) sv[e] = scale2 < 0.f ? 0x7f800000u : 0xff800000u;
  }
  return scale2 == 0.f ? 1.f : scale2;
}

// Clears the rows of a V tile from `row` on: those behind the last token, which may hold anything.  By the
// lanes that loaded the tile, once it has landed; the issuers wait for it.
template <int kCB>
__device__ __forceinline__ void clear_behind(uint8_t* tile, int row, int lane, int lanes) {
  const int n = (kBN - row) * 8;
  for (int x = lane; x < n * kCB; x += lanes) *reinterpret_cast<uint4*>(tile + x / n * 16384 + row * 128 + x % n * 16) = make_uint4(0, 0, 0, 0);
  fence_async_smem();
}

// Whether a row's base (paged.h) may have to move for a tile's largest score; `high`: where it rises.
template <typename T>
__device__ __forceinline__ bool base_off(float m, float high, float top) { return top > high || (kNarrow<T> && top < m - kFall); }
// Moves it to where that score wants it, the row's sum along; returns O's factor.  Only a warp that has such a
// row asks (2048 queries over 32768 tokens: 764 us, all asking 778), in fp16 by a call (796 us, inlined 819).
template <typename T>
__device__ __forceinline__ float3 moved_base(float m, float l, float top) {
  if (!(top > base_high<T>(m)) && !(kNarrow<T> && base_falls(m, top, l))) return make_float3(m, l, 1.f);
  const float to = base_of<T>(top), alpha = ex2(m - to);  // 0 when m was -inf
  return make_float3(to, l * alpha, alpha);
}
__device__ __noinline__ float3 moved_base_half(float m, float l, float top) { return moved_base<__half>(m, l, top); }
template <typename T>
__device__ __forceinline__ float move_base(float& m, float& l, float& high, float top) {
  const float3 x = kNarrow<T> ? moved_base_half(m, l, top) : moved_base<T>(m, l, top);
  m = x.x;
  l = x.y;
  high = base_high<T>(m);
  return x.z;
}

// Maximum of c·s over the keys e < lim of a row of scores; -inf without any.
template <bool kCut>
__device__ __forceinline__ float row_max(const uint32_t (&sv)[kBN], float c, int lim) {
  constexpr int kH = kBN / 2;
  if (kCut && lim <= 0) return minus_inf();
  const float worst = c >= 0.f ? minus_inf() : -minus_inf();
  float acc[4] = {worst, worst, worst, worst};
  if (c >= 0.f) {
#pragma unroll
    for (int e = 0; e < kH; ++e)
      acc[e % 4] = fmax3(acc[e % 4], !kCut || e < lim ? __uint_as_float(sv[e]) : worst, !kCut || kH + e < lim ? __uint_as_float(sv[kH + e]) : worst);
    return fmaxf(fmaxf(acc[0], acc[1]), fmaxf(acc[2], acc[3])) * c;
  }
#pragma unroll
  for (int e = 0; e < kH; ++e)
    acc[e % 4] = fmin3(acc[e % 4], !kCut || e < lim ? __uint_as_float(sv[e]) : worst, !kCut || kH + e < lim ? __uint_as_float(sv[kH + e]) : worst);
  return fminf(fminf(acc[0], acc[1]), fminf(acc[2], acc[3])) * c;
}

// P = 2^(c·s − m) of a row into TMEM, packed in pairs at columns [0, 64), and its sum.  With kSplit
// also what the packing leaves, at columns [64, 128).  `half` is told when the first 64 keys are there.
template <typename T, bool kCut, bool kSplit>
__device__ __forceinline__ float exponentials(const uint32_t (&sv)[kBN], uint32_t s_addr, float c, float neg_m, int lim, uint64_t* half) {
  constexpr int kPiece = kSplit ? 16 : 64;  // keys packed at once
  const uint64_t cc = f2pack(c, c), nm = f2pack(neg_m, neg_m);
  uint64_t acc[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
#pragma unroll
  for (int q = 0; q < kBN / kPiece; ++q) {
    uint32_t pk[kPiece / 2], rest[kPiece / 2];
#pragma unroll
    for (int e = 0; e < kPiece / 2; ++e) {
      const int col = kPiece * q + 2 * e;
      uint64_t x = ffma2(f2pack(__uint_as_float(sv[col]), __uint_as_float(sv[col + 1])), cc, nm);
      if constexpr (kCut) {
        float x0, x1;
        f2unpack(x, x0, x1);
        x = f2pack(col < lim ? x0 : minus_inf(), col + 1 < lim ? x1 : minus_inf());
      }
      float p0, p1;
      ex2_pair(x, p0, p1);
      acc[e % 2] = fadd2(acc[e % 2], f2pack(p0, p1));
      pk[e] = tc::pack2<T>(p0, p1);
      if constexpr (kSplit) {
        float h0, h1;
        unpack2<T>(pk[e], h0, h1);
        rest[e] = tc::pack2<T>(p0 - h0, p1 - h1);
      }
    }
    if constexpr (kSplit) {
      tmem_st8(s_addr + 8 * q, pk);
      tmem_st8(s_addr + 64 + 8 * q, rest);
    } else {
      tmem_st32(s_addr + 32 * q, pk);
      if (q == 0 && half) {
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(half);
      }
    }
  }
  float a, b, d, e;
  f2unpack(acc[0], a, b);
  f2unpack(acc[1], d, e);
  return (a + b) + (d + e);
}

// One row's state at the end: writes its output into the staging tile (or its partial result
// into the workspace) and its logsumexp.  (The staging tile is the Q tile, which nobody reads any more.)
template <typename T, int D>
__device__ __forceinline__ void finish_row(const PagedArgs& a, const Work& w, const Tiling& t, const Rows& rows, const Span& span, int r, uint32_t o_addr,
                                           uint8_t* stage, float m, float l, bool any) {
  const int i = span.i0 + r / t.heads, hq = w.h * a.G + w.group * t.heads + r % t.heads;
  const bool there = r < t.heads * t.tokens && i < span.i1;
  const int lim = there ? rows.limit(i) : 0;
  const int to = min(span.end, lim);
  if (to <= w.k_lo) {  // nothing seen here (what TMEM holds may be anything)
    m = minus_inf();
    l = 0.f;
  }
  const bool nothing = l == 0.f;
  const int64_t row = ((int64_t)w.b * a.Hq + hq) * a.c.L + i;
  float inv = 1.f, m_all = m, l_all = l;
  if (!w.cut && there) {
    const float f = fold_sink(a.sinks, hq, m_all, l_all);
    inv = f / l_all;
    if (a.lse) a.lse[row] = l_all == 0.f ? minus_inf() : (m_all + log2f(l_all)) * kLn2;
  }
  const int64_t at = part_of(t.cut, w.b, a.Hq, hq, i, w.split);
  float* part = a.workspace + at * D;
#pragma unroll 1
  for (int c32 = 0; c32 < D / 32; ++c32) {
    uint32_t o[32];
    if (any) {
      tmem_ld32(o_addr + c32 * 32, o);
      tmem_ld_wait(o);
    }
    bool odd = false;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      if (nothing) o[e] = 0u;
      odd |= (o[e] & 0x7fffffffu) > 0x7f800000u;
    }
    if (odd && l == l) {  // see mend_columns
      float x[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(o[e]);
      mend_columns<T, D, 32>(a, w.b, w.h, hq, i, c32 * 32, w.k_lo, to, m, x);
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(x[e]);
    }
    __syncwarp();
    if (w.cut) {
      if (there && to > w.k_lo)
#pragma unroll
        for (int e = 0; e < 32; e += 4) *reinterpret_cast<uint4*>(part + c32 * 32 + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
    } else {
      uint32_t packed[16];
#pragma unroll
      for (int e = 0; e < 16; ++e)
        packed[e] = nothing ? 0u : tc::pack2<T>(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
      uint8_t* blk = stage + c32 / 2 * 16384;
#pragma unroll
      for (int v4 = 0; v4 < 4; ++v4)
        *reinterpret_cast<uint4*>(blk + sw128_off(r, c32 % 2 * 4 + v4)) = make_uint4(packed[4 * v4], packed[4 * v4 + 1], packed[4 * v4 + 2], packed[4 * v4 + 3]);
    }
  }
  if (w.cut && there && to > w.k_lo) {
    float* ml = part_stats(a, t.cut) + 2 * at;
    ml[0] = m;
    ml[1] = l;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tkv, const __grid_constant__ CUtensorMap to,
                       PagedArgs a, Tiling t) {
  using L = Layout128<D>;
  constexpr int kCB = L::kCB;
  constexpr uint32_t kIdS = idesc_f16(kBM, kBN, kIsBf16<T>, false, false);
  constexpr uint32_t kIdO = idesc_f16(kBM, D, kIsBf16<T>, false, true);
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ unsigned char smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Bars bars;
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Work work = work_of(a, t, 2 * t.tokens);
  const int* table = c.pages + work.b * c.pages_stride;
  // Lane x of the loading warp takes box x / kCB of a tile, column block x % kCB; the first tile's page
  // table entries are on their way while the length is.
  const int boxes = kBN / t.box, box = lane / kCB, cb = lane % kCB;
  Box entry{-1, 0};
  if (warp == kLoadWarp && box < boxes) entry = entry_at(c, table, work.k_lo + box * t.box);
  const Rows rows = rows_of(c, work.b, a.causal, a.max_len, kKidPagedAttn);
  const Span span[2] = {span_of(rows, t, work.i0, work), span_of(rows, t, work.i0 + t.tokens, work)};
  const int nkv[2] = {tiles_in(span[0], work.k_lo), tiles_in(span[1], work.k_lo)};
  const int nmax = max(nkv[0], nkv[1]), end = max(span[0].end, span[1].end);
  const bool tail = nmax > 0 && work.k_lo + nmax * kBN > rows.len;  // the last KV tile holds places behind the last token
  if (nmax == 0 && work.cut) {
    asm volatile("griddepcontrol.launch_dependents;");
    return;
  }
  if (threadIdx.x == 0) {
    bars.abort = 0;
    mbar_init(&bars.q_full, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars.kv_full[s], 1);
      mbar_init(&bars.kv_empty[s], 2);  // both issuers
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bars.s_full[w], 1);
      mbar_init(&bars.p_half[w], kBM);
      mbar_init(&bars.p_full[w], kBM);
      mbar_init(&bars.o_done[w], 1);
      mbar_init(&bars.mma_done[w], 1);
      mbar_init(&bars.turn[w], 4);  // one arrival a warp of the other warpgroup
    }
    mbar_init(&bars.scanned, 1);
    mbar_init(&bars.tail_clean, 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars.tmem_base, 512);
    tmem_relinquish();
  }
  for (int w = 0; w < 2; ++w) clear_unused<kCB>(sm + L::kQOff + w * L::kTileBytes, t);
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bars.tmem_base;
  const WaitCtx wc{&bars.abort, 0, a.wait_limit_ns, c.err, kKidPagedAttn};
  if (warp >= 8) regs_dec<kRegsLow>();

  if (warp == kLoadWarp) {
    if (lane == 0) {
      prefetch_tmap(&tq);
      prefetch_tmap(&tkv);
      prefetch_tmap(&to);
      const int nq = span[1].i0 < c.L ? 2 : 1;
      mbar_arrive_expect_tx(&bars.q_full, nq * kCB * t.heads * t.tokens * 128);
      for (int w = 0; w < nq; ++w)
        for (int cb = 0; cb < kCB; ++cb)
          tma_load_4d(sm + L::kQOff + w * L::kTileBytes + cb * 16384, &tq, &bars.q_full, cb * 64, work.h * a.G + work.group * t.heads, span[w].i0, work.b);
    }
    __syncwarp();
    const bool mine = box < boxes;
    int issued = 0;
    bool ok = true;
    Box at = box_of(c, entry, work.k_lo + box * t.box, mine ? end : 0);
    for (int j = 0; ok && j < nmax; ++j) {
      const Box next = box_at(c, table, work.k_lo + (j + 1) * kBN + box * t.box, mine ? end : 0);
      for (int kv = 0; kv < 2; ++kv) {
        const int it = 2 * j + kv, s = it % kStages;
        ok = __all_sync(kAll, mbar_wait(&bars.kv_empty[s], ((it / kStages) & 1) ^ 1, wc));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bars.kv_full[s], L::kTileBytes);
        __syncwarp();
        if (mine)
          tma_load_4d(sm + L::kRingOff + s * L::kTileBytes + cb * 16384 + box * t.box * 128, &tkv, &bars.kv_full[s], cb * 64, at.place, kv * c.Hkv + work.h, at.page);
        issued = it + 1;
      }
      at = next;
    }
    if (ok && tail) {
      const int it = 2 * nmax - 1;
      if (__all_sync(kAll, mbar_wait(&bars.kv_full[it % kStages], (it / kStages) & 1, wc))) {
        clear_behind<kCB>(sm + L::kRingOff + it % kStages * L::kTileBytes, rows.len - work.k_lo - (nmax - 1) * kBN, lane, 32);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.tail_clean);
      }
    }
    // No copy is in flight when the block exits, whatever its other warps met.
    for (int it = max(0, issued - kStages); it < issued; ++it) drain_wait(&bars.kv_full[it % kStages], (it / kStages) & 1);
    drain_wait(&bars.q_full, 0);
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    const int w = __shfl_sync(kAll, warp - kMmaWarp, 0);
    const int nkv_w = w == 0 ? nkv[0] : nkv[1];
    const bool few = w == 0 ? split_tile(span[0], work.k_lo) : split_tile(span[1], work.k_lo);  // of the first KV tile
    bool ok = __all_sync(kAll, mbar_wait(&bars.q_full, 0, wc));
    tc_fence_after();
    const uint64_t qd = sdesc_sw128(smem_u32(sm + L::kQOff) + w * L::kTileBytes, 16, 1024);
    const uint32_t ring = smem_u32(sm + L::kRingOff);
    const uint32_t s_tm = tbase + w * 128, o_tm = tbase + 256 + w * 128;
    auto scores = [&](int stage) {
      const uint64_t kd = sdesc_sw128(ring + stage * L::kTileBytes, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * 16384 + (kk % 4) * 32;
        mma_ss_w(s_tm, sdesc_advance(qd, off), sdesc_advance(kd, off), kIdS, kk > 0);
      }
    };
    auto values = [&](int stage, int hi, uint32_t p_tm, bool first) {  // keys [64·hi, 64·hi + 64)
      const uint64_t vd = sdesc_sw128(ring + stage * L::kTileBytes, 16384, 1024);
#pragma unroll
      for (int kk = 4 * hi; kk < 4 * hi + 4; ++kk) mma_ts_w(o_tm, p_tm + kk * 8, sdesc_advance(vd, kk * 2048), kIdO, (!first || kk > 0) ? 1u : 0u);
    };
    if (ok && nmax > 0) {
      ok = __all_sync(kAll, mbar_wait(&bars.kv_full[0], 0, wc));
      if (ok && nkv_w > 0) {
        tc_fence_after();
        scores(0);
        mma_commit_w(&bars.s_full[w]);
      }
      if (ok) mma_commit_w(&bars.kv_empty[0]);
    }
    // Every use of a ring stage gets one arrival from each issuer, in order.
    for (int j = 0; ok && j < nmax; ++j) {
      const int itv = 2 * j + 1, itk = 2 * j + 2, sv = itv % kStages, sk = itk % kStages;
      const bool act = j < nkv_w, split = act && j == 0 && few;
      if (!(ok = __all_sync(kAll, mbar_wait(&bars.kv_full[sv], (itv / kStages) & 1, wc)))) break;
      if (act) {
        if (tail && j == nmax - 1 && !(ok = __all_sync(kAll, mbar_wait(&bars.tail_clean, 0, wc)))) break;
        if (!(ok = __all_sync(kAll, mbar_wait(split ? &bars.p_full[w] : &bars.p_half[w], j & 1, wc)))) break;
        tc_fence_after();
        values(sv, 0, s_tm, j == 0);
        if (!split) {
          if (!(ok = __all_sync(kAll, mbar_wait(&bars.p_full[w], j & 1, wc)))) break;
          tc_fence_after();
        }
        values(sv, 1, s_tm, false);
        if (split) {
          values(sv, 0, s_tm + 64, false);
          values(sv, 1, s_tm + 64, false);
        }
        mma_commit_w(&bars.o_done[w]);
      }
      mma_commit_w(&bars.kv_empty[sv]);
      if (j + 1 < nmax) {
        if (!(ok = __all_sync(kAll, mbar_wait(&bars.kv_full[sk], (itk / kStages) & 1, wc)))) break;
        if (j + 1 < nkv_w) {
          if (!(ok = __all_sync(kAll, mbar_wait(&bars.o_done[w], j & 1, wc)))) break;  // P(j) consumed
          tc_fence_after();
          scores(sk);
          mma_commit_w(&bars.s_full[w]);
        }
        mma_commit_w(&bars.kv_empty[sk]);
      }
    }
    mma_commit_w(&bars.mma_done[w]);
    drain_wait(&bars.mma_done[w], 0);
  } else if (warp == kScanWarp) {
    const bool bad = pages_bad(c, table, work.k_lo, end);
    if (lane == 0) {
      bars.bad_pages = bad;
      mbar_arrive(&bars.scanned);
    }
  } else if (warp < 8) {
    regs_inc<kRegsHigh>();
    const int w = warp / 4, quarter = warp % 4, r = quarter * 32 + lane;
    const Span sp = w == 0 ? span[0] : span[1];
    const int mine = w == 0 ? nkv[0] : nkv[1], nboth = min(nkv[0], nkv[1]);
    const uint32_t s_addr = tmem_addr(tbase, quarter * 32, w * 128), o_addr = tmem_addr(tbase, quarter * 32, 256 + w * 128);
    const int i = sp.i0 + r / t.heads;
    const int limit = r < t.heads * t.tokens && i < sp.i1 ? rows.limit(i) : 0;
    float m = minus_inf(), l = 0.f, high = minus_inf();
    bool ok = __all_sync(kAll, mbar_wait(&bars.scanned, 0, wc));
    const bool bad_pages = bars.bad_pages;
    for (int j = 0; ok && j < mine; ++j) {
      const int k0 = work.k_lo + j * kBN;
      if (!(ok = __all_sync(kAll, mbar_wait(&bars.s_full[w], j & 1, wc)))) break;
      tc_fence_after();
      uint32_t sv[kBN];
#pragma unroll
      for (int q4 = 0; q4 < kBN / 32; ++q4) tmem_ld32(s_addr + 32 * q4, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * q4]));
      tmem_ld_wait(sv);
      const bool cut = k0 + kBN > sp.least;
      const int lim = min(limit - k0, kBN);
      float cs = a.scale_log2;
      if (bad_pages) cs = hide_bad_pages(sv, c, table, k0, end, cs);
      const float top = cut ? row_max<true>(sv, cs, lim) : row_max<false>(sv, cs, lim);
      if (__any_sync(kAll, base_off<T>(m, high, top))) {
        const float alpha = move_base<T>(m, l, high, top);
        if (j > 0 && __any_sync(kAll, alpha != 1.f)) {  // rescale O once PV(j-1) has landed
          if (!(ok = __all_sync(kAll, mbar_wait(&bars.o_done[w], (j - 1) & 1, wc)))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c32 = 0; c32 < D / 32; ++c32) {
            uint32_t o[32];
            tmem_ld32(o_addr + c32 * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(o_addr + c32 * 32, o);
          }
          tmem_st_wait();
        }
      }
      if (j < nboth && (w == 1 || j > 0))
        if (!(ok = __all_sync(kAll, mbar_wait(&bars.turn[w], (w == 1 ? j : j - 1) & 1, wc)))) break;
      const float neg_m = m == minus_inf() ? 0.f : -m;  // (nothing seen so far: P = 0 under any finite shift)
      const bool split = j == 0 && split_tile(sp, k0);
      if (split) l += exponentials<T, true, true>(sv, s_addr, cs, neg_m, lim, nullptr);
      else if (cut) l += exponentials<T, true, false>(sv, s_addr, cs, neg_m, lim, &bars.p_half[w]);
      else l += exponentials<T, false, false>(sv, s_addr, cs, neg_m, lim, &bars.p_half[w]);
      tmem_st_wait();
      tc_fence_before();
      if (split) mbar_arrive(&bars.p_half[w]);  // one phase a tile
      // The turn goes to the other tile before P is announced: then no warp's arrival for the next
      // KV tile can count for this one.
      if (j < nboth - w) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.turn[1 - w]);
      }
      mbar_arrive(&bars.p_full[w]);
    }
    if (ok && mine > 0) ok = __all_sync(kAll, mbar_wait(&bars.o_done[w], (mine - 1) & 1, wc));
    // Output rows are staged in the tile's Q buffer, whose last reader has finished.  (A tile
    // without keys may still have its queries on their way.)
    if (ok) ok = __all_sync(kAll, mbar_wait(&bars.q_full, 0, wc));
    if (sp.i0 < c.L) {
      uint8_t* stage = sm + L::kQOff + w * L::kTileBytes;
      if (ok) {
        tc_fence_after();
        finish_row<T, D>(a, work, t, rows, sp, r, o_addr, stage, m, l, mine > 0);
        fence_async_smem();
      }
      if (named_sync_and(1 + w, kBM, ok) && r == 0 && !work.cut) {
        for (int cb = 0; cb < kCB; ++cb) tma_store_4d(&to, stage + cb * 16384, cb * 64, work.h * a.G + work.group * t.heads, sp.i0, work.b);
        bulk_commit();
        bulk_wait_read();
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;");
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_dealloc(tbase, 512);
  }
}

// ---- one Q tile a block
//
// Head dim 256, whose O takes 256 columns of tensor memory (beside two S buffers, so that S of the
// next keys is there while this tile's softmax runs), and calls whose rows all fit in one Q tile
// (drafts, short chunks): then two blocks share an SM, with one S buffer each, and each other's
// waits.  Keys are handed back in blocks of 64 columns and values in halves of 64 tokens, as soon as
// the product that reads them is done with that piece.  Warps 0-3: softmax; warp 4 loads, its first half
// the queries and keys, its second half the values; warp 5 issues S, and PV too where S has one
// buffer (the two take turns then); warp 6 issues PV where it has two.
// `exact`: every tile takes P as head and remainder, so that few rows, whose tiles are bound by the
// bytes of the cache, come out as they do in paged_few.cu.
template <int D>
struct OneLayout {
  static constexpr int kCB = (D + 63) / 64;
  static constexpr int kTileBytes = 128 * kCB * 128;
  static constexpr int kS = D == 256 ? 2 : 1;        // S buffers
  static constexpr int kStages = D <= 64 ? 2 : 1;    // of K tiles and of V tiles
  static constexpr int kKOff = kTileBytes, kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kBytes = kVOff + kStages * kTileBytes + 1024;
  static constexpr int kColumns = D == 256 ? 512 : 256, kO = 128 * kS;
  static constexpr int kThreads = D == 256 ? 256 : 192, kBlocks = D == 256 ? 1 : 2;
};

template <int kCB, int kStages, int kS>
struct OneBars {
  uint64_t q_full, k_full[kStages][kCB], k_empty[kStages][kCB], v_full[kStages][2], v_empty[kStages][2];
  uint64_t s_full[kS], p_full[kS], pv_done[kS], fin, scanned, tail_clean;
  uint32_t tmem_base;
  int abort, bad_pages;
};

template <typename T, int D>
__global__ void __launch_bounds__(OneLayout<D>::kThreads, OneLayout<D>::kBlocks)
    paged_one_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tkv, const __grid_constant__ CUtensorMap to,
                     PagedArgs a, Tiling t, bool exact) {
  using L = OneLayout<D>;
  constexpr int kCB = L::kCB, kS = L::kS, kStages = L::kStages;
  constexpr uint32_t kIdS = idesc_f16(kBM, kBN, kIsBf16<T>, false, false);
  constexpr uint32_t kIdO = idesc_f16(kBM, D, kIsBf16<T>, false, true);
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ unsigned char smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ OneBars<kCB, kStages, kS> bars;
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Work work = work_of(a, t, t.tokens);
  const int* table = c.pages + work.b * c.pages_stride;
  // Lanes 0-15 of the loading warp: box `lane` of each column block of a K tile.  Lanes 16-31: of each
  // half of a V tile, box (lane − 16) / kCB, column block (lane − 16) % kCB.
  const bool loads_k = lane < 16;
  const int box = loads_k ? lane : (lane - 16) / kCB;
  const bool mine = box < (loads_k ? kBN : kBN / 2) / t.box;
  Box entry[2] = {{-1, 0}, {-1, 0}};  // the first K tile's, or both halves' of the first V tile
  if (warp == 4 && mine) {
    entry[0] = entry_at(c, table, work.k_lo + box * t.box);
    if (!loads_k) entry[1] = entry_at(c, table, work.k_lo + kBN / 2 + box * t.box);
  }
  const Rows rows = rows_of(c, work.b, a.causal, a.max_len, kKidPagedAttn);
  const Span span = span_of(rows, t, work.i0, work);
  const int n = tiles_in(span, work.k_lo), end = span.end;
  const bool tail = n > 0 && work.k_lo + n * kBN > rows.len;  // the last KV tile holds places behind the last token
  if (n == 0 && work.cut) {
    asm volatile("griddepcontrol.launch_dependents;");
    return;
  }
  if (threadIdx.x == 0) {
    bars.abort = 0;
    mbar_init(&bars.q_full, 1);
    for (int s = 0; s < kStages; ++s) {
      for (int x = 0; x < kCB; ++x) {
        mbar_init(&bars.k_full[s][x], 1);
        mbar_init(&bars.k_empty[s][x], 1);
      }
      for (int x = 0; x < 2; ++x) {
        mbar_init(&bars.v_full[s][x], 1);
        mbar_init(&bars.v_empty[s][x], 1);
      }
    }
    for (int x = 0; x < kS; ++x) {
      mbar_init(&bars.s_full[x], 1);
      mbar_init(&bars.p_full[x], kBM);
      mbar_init(&bars.pv_done[x], 1);
    }
    mbar_init(&bars.fin, kS);  // one commit an issuer
    mbar_init(&bars.scanned, 1);
    mbar_init(&bars.tail_clean, 1);
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(&bars.tmem_base, L::kColumns);
    tmem_relinquish();
  }
  clear_unused<kCB>(sm, t);
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bars.tmem_base;
  const WaitCtx wc{&bars.abort, 0, a.wait_limit_ns, c.err, kKidPagedAttn};
  const auto few = [&](int j) { return exact || (j == 0 && split_tile(span, work.k_lo)); };

  if (warp == 4) {
    const unsigned half = loads_k ? 0x0000ffffu : 0xffff0000u;
    const bool first = lane % 16 == 0;
    bool ok = true;
    int issued = 0;  // pieces
    if (lane == 0) {
      prefetch_tmap(&tq);
      prefetch_tmap(&tkv);
      prefetch_tmap(&to);
      mbar_arrive_expect_tx(&bars.q_full, kCB * t.heads * t.tokens * 128);
      for (int cb = 0; cb < kCB; ++cb) tma_load_4d(sm + cb * 16384, &tq, &bars.q_full, cb * 64, work.h * a.G + work.group * t.heads, work.i0, work.b);
    }
    __syncwarp();
    if (loads_k) {
      Box at = box_of(c, entry[0], work.k_lo + box * t.box, mine ? end : 0);
      for (int j = 0; ok && j < n; ++j) {
        const int s = j % kStages;
        const Box next = box_at(c, table, work.k_lo + (j + 1) * kBN + box * t.box, mine ? end : 0);
        for (int cb = 0; cb < kCB; ++cb) {
          if (!(ok = __all_sync(half, mbar_wait(&bars.k_empty[s][cb], ((j / kStages) & 1) ^ 1, wc)))) break;
          if (first) mbar_arrive_expect_tx(&bars.k_full[s][cb], kBN * 128);
          __syncwarp(half);
          if (mine)
            tma_load_4d(sm + L::kKOff + s * L::kTileBytes + cb * 16384 + box * t.box * 128, &tkv, &bars.k_full[s][cb], cb * 64, at.place, work.h, at.page);
          ++issued;
        }
        at = next;
      }
      // No copy is in flight when the block exits, whatever its other warps met.
      for (int x = max(0, issued - kStages * kCB); x < issued; ++x) drain_wait(&bars.k_full[x / kCB % kStages][x % kCB], (x / kCB / kStages) & 1);
      drain_wait(&bars.q_full, 0);
    } else {
      const int cb = (lane - 16) % kCB;
      Box at[2];
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) at[hr] = box_of(c, entry[hr], work.k_lo + hr * (kBN / 2) + box * t.box, mine ? end : 0);
      for (int j = 0; ok && j < n; ++j) {
        const int s = j % kStages;
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          const Box next = box_at(c, table, work.k_lo + (j + 1) * kBN + hr * (kBN / 2) + box * t.box, mine ? end : 0);
          if (ok && (ok = __all_sync(half, mbar_wait(&bars.v_empty[s][hr], ((j / kStages) & 1) ^ 1, wc)))) {
            if (first) mbar_arrive_expect_tx(&bars.v_full[s][hr], L::kTileBytes / 2);
            __syncwarp(half);
            if (mine)
              tma_load_4d(sm + L::kVOff + s * L::kTileBytes + cb * 16384 + (hr * (kBN / 2) + box * t.box) * 128, &tkv, &bars.v_full[s][hr], cb * 64, at[hr].place,
                          c.Hkv + work.h, at[hr].page);
            ++issued;
          }
          at[hr] = next;
        }
      }
      if (ok && tail) {
        const int s = (n - 1) % kStages, ph = ((n - 1) / kStages) & 1;
        if (__all_sync(half, mbar_wait(&bars.v_full[s][0], ph, wc) && mbar_wait(&bars.v_full[s][1], ph, wc))) {
          clear_behind<kCB>(sm + L::kVOff + s * L::kTileBytes, rows.len - work.k_lo - (n - 1) * kBN, lane - 16, 16);
          __syncwarp(half);
          if (first) mbar_arrive(&bars.tail_clean);
        }
      }
      for (int x = max(0, issued - kStages * 2); x < issued; ++x) drain_wait(&bars.v_full[x / 2 % kStages][x % 2], (x / 2 / kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 5 || (kS == 2 && warp == 6)) {
    const bool s_issuer = __shfl_sync(kAll, warp, 0) == 5, pv_issuer = kS == 1 || !s_issuer;
    if (s_issuer) {
      const bool bad = pages_bad(c, table, work.k_lo, end);
      if (lane == 0) {
        bars.bad_pages = bad;
        mbar_arrive(&bars.scanned);
      }
    }
    bool ok = __all_sync(kAll, mbar_wait(&bars.q_full, 0, wc));
    tc_fence_after();
    const uint64_t qd = sdesc_sw128(smem_u32(sm), 16, 1024);
    auto scores = [&](int j) {
      const int s = j % kStages, buf = j % kS;
      const uint64_t kd = sdesc_sw128(smem_u32(sm + L::kKOff + s * L::kTileBytes), 16, 1024);
#pragma unroll
      for (int cb = 0; cb < kCB; ++cb) {
        if (!(ok = __all_sync(kAll, mbar_wait(&bars.k_full[s][cb], (j / kStages) & 1, wc)))) return;
        tc_fence_after();
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
          if (cb * 4 + k4 < D / 16) mma_ss_w(tbase + 128 * buf, sdesc_advance(qd, cb * 16384 + k4 * 32), sdesc_advance(kd, cb * 16384 + k4 * 32), kIdS, cb + k4 > 0);
        mma_commit_w(&bars.k_empty[s][cb]);
      }
      mma_commit_w(&bars.s_full[buf]);
    };
    auto values = [&](int j) {
      const int s = j % kStages, buf = j % kS;
      if (!(ok = __all_sync(kAll, mbar_wait(&bars.p_full[buf], (j / kS) & 1, wc)))) return;
      const uint64_t vd = sdesc_sw128(smem_u32(sm + L::kVOff + s * L::kTileBytes), 16384, 1024);
      const uint32_t p_tm = tbase + 128 * buf;
      const bool split = few(j);
      if (tail && j == n - 1 && !(ok = __all_sync(kAll, mbar_wait(&bars.tail_clean, 0, wc)))) return;
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        if (!(ok = __all_sync(kAll, mbar_wait(&bars.v_full[s][hr], (j / kStages) & 1, wc)))) return;
        tc_fence_after();
#pragma unroll
        for (int kk = 4 * hr; kk < 4 * hr + 4; ++kk) mma_ts_w(tbase + L::kO, p_tm + kk * 8, sdesc_advance(vd, kk * 2048), kIdO, (j > 0 || kk > 0) ? 1u : 0u);
        if (split) {
#pragma unroll
          for (int kk = 4 * hr; kk < 4 * hr + 4; ++kk) mma_ts_w(tbase + L::kO, p_tm + 64 + kk * 8, sdesc_advance(vd, kk * 2048), kIdO, 1u);
        }
        mma_commit_w(&bars.v_empty[s][hr]);
      }
      mma_commit_w(&bars.pv_done[buf]);
    };
    if constexpr (kS == 1) {
      if (ok && n > 0) scores(0);
      for (int j = 0; ok && j < n; ++j) {
        values(j);
        if (!ok || j + 1 == n) break;
        if (!(ok = __all_sync(kAll, mbar_wait(&bars.pv_done[0], j & 1, wc)))) break;  // P(j) consumed
        tc_fence_after();
        scores(j + 1);
      }
    } else {
      for (int j = 0; ok && j < n; ++j) {
        if (pv_issuer) {
          values(j);
        } else {
          if (j >= 2 && !(ok = __all_sync(kAll, mbar_wait(&bars.pv_done[j % 2], ((j - 2) / 2) & 1, wc)))) break;
          tc_fence_after();
          scores(j);
        }
      }
    }
    mma_commit_w(&bars.fin);
    drain_wait(&bars.fin, 0);
  } else if (warp < 4) {
    const int r = warp * 32 + lane;
    const uint32_t o_addr = tmem_addr(tbase, warp * 32, L::kO);
    const int i = span.i0 + r / t.heads;
    const int limit = r < t.heads * t.tokens && i < span.i1 ? rows.limit(i) : 0;
    const bool live = __any_sync(kAll, limit > 0);  // a warp without a row only keeps the barriers going
    float m = minus_inf(), l = 0.f, high = minus_inf();
    bool ok = __all_sync(kAll, mbar_wait(&bars.scanned, 0, wc));
    const bool bad_pages = bars.bad_pages;
    for (int j = 0; ok && j < n; ++j) {
      const int k0 = work.k_lo + j * kBN, buf = j % kS;
      if (!(ok = __all_sync(kAll, mbar_wait(&bars.s_full[buf], (j / kS) & 1, wc)))) break;
      tc_fence_after();
      if (live) {
        const uint32_t s_addr = tmem_addr(tbase, warp * 32, 128 * buf);
        uint32_t sv[kBN];
#pragma unroll
        for (int q4 = 0; q4 < kBN / 32; ++q4) tmem_ld32(s_addr + 32 * q4, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * q4]));
        tmem_ld_wait(sv);
        const bool cut = k0 + kBN > span.least;
        const int lim = min(limit - k0, kBN);
        float cs = a.scale_log2;
        if (bad_pages) cs = hide_bad_pages(sv, c, table, k0, end, cs);
        const float top = cut ? row_max<true>(sv, cs, lim) : row_max<false>(sv, cs, lim);
        if (__any_sync(kAll, base_off<T>(m, high, top))) {
          const float alpha = move_base<T>(m, l, high, top);
          if (j > 0 && __any_sync(kAll, alpha != 1.f)) {  // rescale O once PV(j-1) has landed
            if (!(ok = __all_sync(kAll, mbar_wait(&bars.pv_done[(j - 1) % kS], ((j - 1) / kS) & 1, wc)))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c32 = 0; c32 < D / 32; ++c32) {
              uint32_t o[32];
              tmem_ld32(o_addr + c32 * 32, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(o_addr + c32 * 32, o);
            }
            tmem_st_wait();
          }
        }
        const float neg_m = m == minus_inf() ? 0.f : -m;
        if (few(j)) l += exponentials<T, true, true>(sv, s_addr, cs, neg_m, lim, nullptr);
        else if (cut) l += exponentials<T, true, false>(sv, s_addr, cs, neg_m, lim, nullptr);
        else l += exponentials<T, false, false>(sv, s_addr, cs, neg_m, lim, nullptr);
        tmem_st_wait();
      }
      tc_fence_before();
      mbar_arrive(&bars.p_full[buf]);
    }
    if (ok && n > 0) ok = __all_sync(kAll, mbar_wait(&bars.pv_done[(n - 1) % kS], ((n - 1) / kS) & 1, wc));
    if (ok) ok = __all_sync(kAll, mbar_wait(&bars.q_full, 0, wc));
    if (ok) {
      tc_fence_after();
      finish_row<T, D>(a, work, t, rows, span, r, o_addr, sm, m, l, n > 0);
      fence_async_smem();
    }
    if (named_sync_and(1, kBM, ok) && r == 0 && !work.cut) {
      for (int cb = 0; cb < kCB; ++cb) tma_store_4d(&to, sm + cb * 16384, cb * 64, work.h * a.G + work.group * t.heads, work.i0, work.b);
      bulk_commit();
      bulk_wait_read();
    }
  }
  asm volatile("griddepcontrol.launch_dependents;");
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    __syncwarp();
    tmem_dealloc(tbase, L::kColumns);
  }
}

// ---- host

template <typename T, int D>
cudaError_t chunk_d(const PagedArgs& a, cudaStream_t s) {
  const Tiling t = paged_tiling(a);
  CUtensorMap tq, tkv, to;
  if (!make_tmap_rows(&tq, a.q, a, a.lq, t) || !make_tmap_rows(&to, a.out, a, a.lo, t) || !make_tmap_pages(&tkv, a.c, t.box)) return cudaErrorInvalidValue;
  if (t.tiles == 1) {
    using L = OneLayout<D>;
    auto* kern = paged_one_kernel<T, D>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(kern, L::kBytes, ready);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)paged_chunk_blocks(a), L::kThreads, L::kBytes, s>>>(tq, tkv, to, a, t, a.G * (int64_t)a.c.L <= 32);
    return cudaGetLastError();
  }
  if constexpr (D <= 128) {
    auto* kern = paged_chunk_kernel<T, D>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(kern, Layout128<D>::kBytes, ready);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)paged_chunk_blocks(a), kThreads, Layout128<D>::kBytes, s>>>(tq, tkv, to, a, t);
    return cudaGetLastError();
  }
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t chunk_t(const PagedArgs& a, cudaStream_t s) {
  switch (a.c.D) {
    case 32: return chunk_d<T, 32>(a, s);
    case 64: return chunk_d<T, 64>(a, s);
    case 96: return chunk_d<T, 96>(a, s);
    case 128: return chunk_d<T, 128>(a, s);
    case 256: return chunk_d<T, 256>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

// The split of the heads that share a KV head into tiles that takes the fewest tiles; of equal
// ones the one with the most heads, whose rows end closest together.
tc::Tiling paged_tiling(const PagedArgs& a) {
  tc::Tiling t = {};
  int64_t best = INT64_MAX;
  for (int heads = min(a.G, tc::kBM); heads >= 1; --heads) {
    if (a.G % heads) continue;
    const int tokens = tc::kBM / heads;
    const int64_t tiles = (int64_t)(a.G / heads) * ((a.c.L + tokens - 1) / tokens);
    if (tiles < best) {
      best = tiles;
      t.heads = heads;
      t.tokens = tokens;
    }
  }
  t.groups = a.G / t.heads;
  t.tiles = a.c.D == 256 || (t.groups == 1 && a.c.L <= t.tokens) ? 1 : 2;
  const int queries = t.tiles * t.tokens;
  t.blocks = (a.c.L + queries - 1) / queries;
  t.box = t.tiles == 1 ? 64 : 128;
  while (a.c.page_size % t.box) t.box /= 2;
  t.whole = t.blocks;
  t.cut = Cut{1 << 30, 1, 0};
  // What does not fill a wave of blocks (one an SM) is cut into chunks of keys, if that is expected
  // to pay: in microseconds, a pair of tiles takes 1.6 a KV tile, a block 4 more, and the join 4 and
  // its bytes at 2.5 TB/s.  Where the causal mask lets queries differ much in what they see, whole waves
  // end evenly anyway.  (The size of the workspace goes by this, and is asked for without the mask.)
  const int64_t units = (int64_t)a.c.B * a.c.Hkv * t.groups, all = units * t.blocks;
  const int64_t sms = (a.c.num_sms > 0 ? a.c.num_sms : 1) * (t.tiles == 1 && a.c.D <= 128 ? 2 : 1);
  const int tiles = (a.max_len + tc::kBN - 1) / tc::kBN;
  const bool even = (int64_t)2 * (a.max_len - a.c.L + queries) >= a.max_len;
  if (all >= sms && !even) return t;
  const int whole = t.blocks == 1 ? 0 : (int)(all / sms * sms / units);
  const int64_t rest = units * (t.blocks - whole);
  const int rows = min(a.c.L, (t.blocks - whole) * queries);
  const double partial = (double)a.c.B * a.Hq * rows * (a.c.D + 2) * sizeof(float);
  double best_time = 1e30;
  int splits = 1;
  for (int x = 1; x <= 64 && (x == 1 || (x * partial <= 67108864.0 && x * 4 <= tiles)); ++x) {
    const double time = (double)((rest * x + sms - 1) / sms) * ((tiles + x - 1) / x * 1.6 + 4) + (x > 1 ? 4 + 2 * x * partial / 2.5e6 : 0);
    if (time < best_time) {
      best_time = time;
      splits = x;
    }
  }
  const int chunk = (tiles + splits - 1) / splits * tc::kBN;
  splits = (a.max_len + chunk - 1) / chunk;
  if (splits > 1) {
    t.whole = whole;
    t.cut = Cut{chunk, splits, rows};
  }
  return t;
}

bool paged_chunk_takes(const PagedArgs& a) { return a.G * (int64_t)a.c.L > (a.c.D == 256 ? 16 : 32); }
Cut paged_chunk_cut(const PagedArgs& a) { return paged_tiling(a).cut; }
int64_t paged_chunk_blocks(const PagedArgs& a) {
  const tc::Tiling t = paged_tiling(a);
  return (int64_t)a.c.B * a.c.Hkv * t.groups * (t.whole + (int64_t)(t.blocks - t.whole) * t.cut.splits);
}
cudaError_t launch_paged_chunk(const PagedArgs& a, int dtype, cudaStream_t s) {
  return dtype == 1 ? chunk_t<__half>(a, s) : chunk_t<__nv_bfloat16>(a, s);
}

}  // namespace sdpa
