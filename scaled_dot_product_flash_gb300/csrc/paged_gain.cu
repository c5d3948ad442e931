// The attention weight that cached tokens gather from many query rows: TMA + tcgen05 + TMEM
// (conventions in include/sdpa.h; few rows: paged_few.cu).
//
// The product is transposed, S^T = K·Q^T with keys as its 128 rows, so that a thread has one key
// and its sum over the queries never leaves the thread: no shuffles, no atomics, one order.  A block
// has KT tiles of 128 keys of one KV head in shared memory for good and streams the Q tiles that see
// them (rows as in paged_tc.cuh) and their logsumexps through a ring.  Eight warps a key tile take
// 2^(c·s − lse) from two TMEM buffers a tile, filled in turn; three more load Q, issue the MMAs, and
// fetch the logsumexps, negated and in units of log2.  Where there are few blocks a
// cluster shares the Q tiles of its keys and adds its sums up in the order of its ranks.
//
// Rows without weight (padding, an lse of −inf, rows that a tile does not fill) have a logsumexp
// of +inf here; since their products may be NaN, the 32-row pieces that hold some are marked, and
// there those terms are left out one by one.
//
// Bound: tensor pipe and exponential unit alike, 512 cycles a pair of 128 x 128 tiles at D = 128.  Measured
// (bf16, 32 query and 8 KV heads, D = 128, from a graph): prompts of 4096 tokens 140 us, both units 44%
// busy; with four warps a key tile 151, and 169 with divisions in the warp that fetches logsumexps, whose
// steps the others wait for.
#include <cooperative_groups.h>

#include "paged_tc.cuh"

namespace sdpa {
namespace {
using namespace tc;
namespace cg = cooperative_groups;

template <int D>
struct GainLayout {
  static constexpr int kCB = (D + 63) / 64;
  static constexpr int kTileBytes = 128 * kCB * 128;
  static constexpr int KT = D == 256 ? 1 : 2;      // key tiles of a block
  static constexpr int kStages = D == 256 ? 2 : 4;  // Q tiles in the ring
  static constexpr int kRingOff = KT * kTileBytes;
  // Eight warps a key tile: four of its keys' quarters, twice, for the halves of the rows.
  static constexpr int kLoadWarp = 8 * KT, kMmaWarp = kLoadWarp + 1, kLseWarp = kLoadWarp + 2;
  static constexpr int kThreads = 32 * (kLoadWarp + 3);
  static constexpr int kBytes = kRingOff + kStages * kTileBytes + 1024;
};

template <int KT, int kStages>
struct GainBars {
  uint64_t k_full, q_full[kStages], q_empty[kStages], lse_full[kStages], lse_empty[kStages];
  uint64_t acc_full[KT][2], acc_empty[KT][2], mma_done;
  alignas(16) float lse[kStages][kBM];  // −lse·log2(e) of the rows, −inf for those without weight
  int dead[kStages];        // bit p: rows [32p, 32p + 32) hold some of those
  float sums[KT][2][kBN];   // of each half of the rows
  uint32_t tmem_base;
  int abort;
};

// A Q tile: its first query and its group of heads; each role steps through the block's tiles by itself.
struct Tile {
  int i0, group, step_i, step_group;
  __device__ __forceinline__ void next(const Tiling& t) {
    i0 += step_i;
    group += step_group;
    if (group >= t.groups) {
      group -= t.groups;
      i0 += t.tokens;
    }
  }
};

// Σ 2^(c·s + x) over 32 rows of one key; rows e < from are hidden.
template <bool kCut, bool kDead>
__device__ __forceinline__ void add_weights(uint64_t (&acc)[2], const uint32_t (&s)[32], const float* x, float c, int from) {
  const uint64_t cc = f2pack(c, c);
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const float4 y = *reinterpret_cast<const float4*>(x + e);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float y0 = h ? y.z : y.x, y1 = h ? y.w : y.y;
      const int at = e + 2 * h;
      float p0, p1;
      ex2_pair(ffma2(f2pack(__uint_as_float(s[at]), __uint_as_float(s[at + 1])), cc, f2pack(y0, y1)), p0, p1);
      if ((kCut && at < from) || (kDead && y0 == minus_inf())) p0 = 0.f;
      if ((kCut && at + 1 < from) || (kDead && y1 == minus_inf())) p1 = 0.f;
      acc[h] = fadd2(acc[h], f2pack(p0, p1));
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(GainLayout<D>::kThreads, 1)
    paged_gain_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tkv, PagedArgs a, Tiling t) {
  using L = GainLayout<D>;
  constexpr int kCB = L::kCB, KT = L::KT, kStages = L::kStages;
  constexpr uint32_t kId = idesc_f16(kBN, kBM, kIsBf16<T>, false, false);
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ unsigned char smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ GainBars<KT, kStages> bars;
  const cg::cluster_group cluster = cg::this_cluster();
  const int cl = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // Grid: (cluster · sequences · KV heads, blocks of keys): the first keys, which most rows see, first.
  const int unit = blockIdx.x / cl, b = unit / c.Hkv, h = unit % c.Hkv;
  const int64_t k_first = (int64_t)blockIdx.y * KT * kBN;
  const Rows rows = rows_of(c, b, a.causal, a.max_len, kKidPagedWeights);
  if (k_first >= rows.len || rows.first >= c.L) return;  // the whole cluster: no keys, or no real row
  const int k0 = (int)k_first, off = rows.len - c.L;      // row i has position off + i
  // Q tiles: blocks of `tokens` queries from the first one that sees the first key, all groups of heads.
  const int i_first = a.causal ? max(rows.first, k0 - off) : rows.first;
  const int t_first = i_first / t.tokens, t_last = (c.L - 1) / t.tokens;
  const int n_all = (t_last - t_first + 1) * t.groups;
  const int n = n_all > me ? (n_all - me + cl - 1) / cl : 0;  // of this block: me, me + cl, ...
  Tile tile{(t_first + me / t.groups) * t.tokens, me % t.groups, cl / t.groups * t.tokens, cl % t.groups};

  if (threadIdx.x == 0) {
    bars.abort = 0;
    mbar_init(&bars.k_full, 1);
    mbar_init(&bars.mma_done, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars.q_full[s], 1);
      mbar_init(&bars.q_empty[s], 1);
      mbar_init(&bars.lse_full[s], 32);
      mbar_init(&bars.lse_empty[s], 8 * KT);
    }
    for (int w = 0; w < KT; ++w)
      for (int x = 0; x < 2; ++x) {
        mbar_init(&bars.acc_full[w][x], 1);
        mbar_init(&bars.acc_empty[w][x], 8);
      }
    fence_mbar_init();
  }
  if (warp == L::kMmaWarp) {
    tmem_alloc(&bars.tmem_base, 512);
    tmem_relinquish();
  }
  for (int s = 0; s < kStages; ++s) clear_unused<kCB>(sm + L::kRingOff + s * L::kTileBytes, t);
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bars.tmem_base;
  const int* table = c.pages + b * c.pages_stride;
  const WaitCtx wc{&bars.abort, 0, a.wait_limit_ns, c.err, kKidPagedWeights};

  if (warp == L::kLoadWarp) {
    if (lane == 0) {
      prefetch_tmap(&tq);
      prefetch_tmap(&tkv);
      mbar_arrive_expect_tx(&bars.k_full, KT * L::kTileBytes);
    }
    __syncwarp();
    const int boxes = KT * kBN / t.box;
    for (int x = lane; x < boxes * kCB; x += 32) {
      const int box = x / kCB, cb = x % kCB, row = box * t.box;
      const Box at = box_at(c, table, k0 + row, rows.len);
      if (k0 + row < rows.len && at.page == c.num_pages) report_error(c.err, kDevErrIndex, kKidPagedWeights);
      tma_load_4d(sm + row / kBN * L::kTileBytes + cb * 16384 + row % kBN * 128, &tkv, &bars.k_full, cb * 64, at.place, h, at.page);
    }
    int issued = 0;
    bool ok = true;
    for (int x = 0; ok && x < n; ++x) {
      const int s = x % kStages;
      ok = __all_sync(kAll, mbar_wait(&bars.q_empty[s], ((x / kStages) & 1) ^ 1, wc));
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&bars.q_full[s], kCB * t.heads * t.tokens * 128);
      __syncwarp();
      if (lane < kCB)
        tma_load_4d(sm + L::kRingOff + s * L::kTileBytes + lane * 16384, &tq, &bars.q_full[s], lane * 64, h * a.G + tile.group * t.heads, tile.i0, b);
      tile.next(t);
      issued = x + 1;
    }
    // No copy is in flight when the block exits, whatever its other warps met.
    drain_wait(&bars.k_full, 0);
    for (int x = max(0, issued - kStages); x < issued; ++x) drain_wait(&bars.q_full[x % kStages], (x / kStages) & 1);
  } else if (warp == L::kMmaWarp) {
    bool ok = __all_sync(kAll, mbar_wait(&bars.k_full, 0, wc));
    tc_fence_after();
    const uint64_t kd = sdesc_sw128(smem_u32(sm), 16, 1024);
    const uint32_t ring = smem_u32(sm + L::kRingOff);
    for (int x = 0; ok && x < n; ++x) {
      const int s = x % kStages, buf = x % 2;
      if (!(ok = __all_sync(kAll, mbar_wait(&bars.q_full[s], (x / kStages) & 1, wc)))) break;
      const uint64_t qd = sdesc_sw128(ring + s * L::kTileBytes, 16, 1024);
#pragma unroll
      for (int w = 0; w < KT; ++w) {
        if (!(ok = __all_sync(kAll, mbar_wait(&bars.acc_empty[w][buf], ((x / 2) & 1) ^ 1, wc)))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t at = (kk / 4) * 16384 + (kk % 4) * 32;
          mma_ss_w(tbase + (2 * w + buf) * kBM, sdesc_advance(kd, w * L::kTileBytes + at), sdesc_advance(qd, at), kId, kk > 0);
        }
        mma_commit_w(&bars.acc_full[w][buf]);
      }
      if (!ok) break;
      mma_commit_w(&bars.q_empty[s]);
    }
    mma_commit_w(&bars.mma_done);
    drain_wait(&bars.mma_done, 0);
  } else if (warp == L::kLseWarp) {
    // Four rows a lane; the next tile's are fetched while this one's wait for their stage.
    float v[kBM / 32];
    int token[kBM / 32];
    const float* from[kBM / 32];  // the row's logsumexps, of the first tile's group and query 0
#pragma unroll
    for (int e = 0; e < kBM / 32; ++e) {
      const int r = 32 * e + lane;
      token[e] = r < t.heads * t.tokens ? r / t.heads : c.L;
      from[e] = a.lse + ((int64_t)b * a.Hq + h * a.G + r % t.heads) * c.L;
    }
    auto fetch = [&] {
#pragma unroll
      for (int e = 0; e < kBM / 32; ++e) {
        const int i = tile.i0 + token[e];
        v[e] = i < c.L && i >= rows.first ? from[e][(int64_t)tile.group * t.heads * c.L + i] : minus_inf();
      }
      tile.next(t);
    };
    if (n > 0) fetch();
    bool ok = true;
    for (int x = 0; ok && x < n; ++x) {
      const int s = x % kStages;
      float y[kBM / 32];
      int dead = 0;
#pragma unroll
      for (int e = 0; e < kBM / 32; ++e) {
        const bool none = v[e] == minus_inf();
        y[e] = none ? minus_inf() : -v[e] * kLog2e;
        dead |= __any_sync(kAll, none) ? 1 << e : 0;
      }
      if (x + 1 < n) fetch();
      if (!(ok = __all_sync(kAll, mbar_wait(&bars.lse_empty[s], ((x / kStages) & 1) ^ 1, wc)))) break;
#pragma unroll
      for (int e = 0; e < kBM / 32; ++e) bars.lse[s][32 * e + lane] = y[e];
      if (lane == 0) bars.dead[s] = dead;
      mbar_arrive(&bars.lse_full[s]);
    }
  } else {
    const int w = warp / 8, half = warp / 4 % 2, quarter = warp % 4, r = quarter * 32 + lane;
    const int key = k0 + w * kBN + r;
    const uint32_t at = tmem_addr(tbase, quarter * 32, 2 * w * kBM);
    uint64_t acc[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
    bool ok = true;
    for (int x = 0; x < n; ++x) {
      const int s = x % kStages, buf = x % 2, i0 = tile.i0;
      tile.next(t);
      ok = __all_sync(kAll, mbar_wait(&bars.lse_full[s], (x / kStages) & 1, wc) && mbar_wait(&bars.acc_full[w][buf], (x / 2) & 1, wc));
      if (!ok) break;
      tc_fence_after();
      // Row r sees the key if off + i0 + r / heads >= key, that is from row (key − off − i0)·heads on.
      const bool cut = a.causal && off + i0 < k0 + w * kBN + kBN - 1;
      const int from = cut ? min(max(key - off - i0, 0), kBM) * t.heads : 0;
      const int dead = bars.dead[s];
#pragma unroll
      for (int x2 = 0; x2 < 2; ++x2) {
        const int p = 2 * half + x2;  // rows [32p, 32p + 32)
        uint32_t sv[32];
        tmem_ld32(at + buf * kBM + 32 * p, sv);
        tmem_ld_wait(sv);
        if (x2 == 1) {  // the scores are in registers: the buffer may be filled again
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.acc_empty[w][buf]);
        }
        const float* y = bars.lse[s] + 32 * p;
        if (dead >> p & 1) add_weights<true, true>(acc, sv, y, a.scale_log2, from - 32 * p);
        else if (cut) add_weights<true, false>(acc, sv, y, a.scale_log2, from - 32 * p);
        else add_weights<false, false>(acc, sv, y, a.scale_log2, 0);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.lse_empty[s]);
    }
    float p0, p1, p2, p3;
    f2unpack(acc[0], p0, p1);
    f2unpack(acc[1], p2, p3);
    bars.sums[w][half][r] = (p0 + p1) + (p2 + p3);
  }
  tc_fence_before();
  cluster.sync();  // (a cluster of one: the block's barrier)
  if (warp == L::kMmaWarp) tmem_dealloc(tbase, 512);
  if (me == 0)
    for (int x = threadIdx.x; x < KT * kBN; x += L::kThreads) {
      const int key = k0 + x;
      if (key >= rows.len) break;
      float sum = 0.f;
      for (int p = 0; p < cl; ++p) {
        const float* y = cluster.map_shared_rank(&bars.sums[x / kBN][0][x % kBN], p);
        sum += y[0] + y[kBN];
      }
      if ((unsigned)table[key / c.page_size] >= (unsigned)c.num_pages) sum = 0.f;  // its page is bad
      float* to = a.weights + b * a.w_batch + h * a.w_head + key;
      *to = (key >= off + rows.first ? 0.f : *to) + sum;
    }
  cluster.sync();  // no block leaves while its sums are being read
}

template <typename T, int D>
cudaError_t gain_d(const PagedArgs& a, cudaStream_t s) {
  using L = GainLayout<D>;
  const Tiling t = paged_tiling(a);
  CUtensorMap tq, tkv;
  if (!make_tmap_rows(&tq, a.q, a, a.lq, t) || !make_tmap_pages(&tkv, a.c, t.box)) return cudaErrorInvalidValue;
  auto* kern = paged_gain_kernel<T, D>;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(kern, L::kBytes, ready);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)a.c.B * a.c.Hkv, blocks = (a.max_len + L::KT * kBN - 1) / (L::KT * kBN);
  const int64_t q_tiles = (int64_t)t.groups * ((a.c.L + t.tokens - 1) / t.tokens);
  // Blocks for two waves and more, so that under the causal mask, where the first keys have the most
  // rows, they end together; at least 8 Q tiles each.
  int cl = 1;
  while (cl < 8 && units * blocks * cl < 2 * (int64_t)a.c.num_sms && cl * 16 <= q_tiles) cl *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * cl), (unsigned)blocks);
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cl;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tq, tkv, a, t);
}

template <typename T>
cudaError_t gain_t(const PagedArgs& a, cudaStream_t s) {
  switch (a.c.D) {
    case 32: return gain_d<T, 32>(a, s);
    case 64: return gain_d<T, 64>(a, s);
    case 96: return gain_d<T, 96>(a, s);
    case 128: return gain_d<T, 128>(a, s);
    case 256: return gain_d<T, 256>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

bool paged_gain_takes(const PagedArgs& a) {
  // (the second dimension of a grid holds 65535 blocks)
  return a.G * (int64_t)a.c.L > 32 && a.max_len <= 65535 * kBN;
}
cudaError_t launch_paged_gain(const PagedArgs& a, int dtype, cudaStream_t s) {
  return dtype == 1 ? gain_t<__half>(a, s) : gain_t<__nv_bfloat16>(a, s);
}

}  // namespace sdpa
