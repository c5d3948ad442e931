// Writing a 16-bit paged cache, and evicting the tokens that have gathered the least attention
// weight (conventions in include/sdpa.h).
//
// Write: every thread moves four 16-byte pieces.  Bound: HBM for prompts, latency for tokens.
//
// Evict, two kernels:
//  - select: a cluster of blocks takes one row of weights (one sequence and KV head).  Weights are
//    ranked as 32-bit keys in their order; three histograms of 11, 11 and 10 bits, summed over the
//    cluster through distributed shared memory, give the key of the last token that stays, and
//    counts of what lies before each token (ballots in a warp, then warps, then blocks) its new place.
//  - move: kept[r] >= r and both ascend, so a block that loads rows in order and stores them only
//    when all of its loads have landed never overwrites a row that is still to be read.  Rows are cut
//    into slices of 32 bytes or more, one block each: slices do not touch one another, and there are
//    enough of them to fill the device.
#include <cooperative_groups.h>

#include "paged.h"

namespace sdpa {
namespace {

namespace cg = cooperative_groups;

constexpr int kWriteThreads = 256, kWriteEach = 4;

template <int D>
__global__ void __launch_bounds__(kWriteThreads) paged_write_kernel(CacheArgs c) {
  constexpr int U = D / 8;  // 16-byte pieces of a row
  const int b = blockIdx.y;
  const int table = c.pages_per_seq * c.page_size;
  const int len = cache_len(c, b, table, kKidPagedWrite);
  // (a sequence whose length lies past the table's end keeps its rows' positions)
  const int n = max(c.lens[b], 0);
  const int count = c.counts ? min(max(c.counts[b], 0), c.L) : c.L;
  const int rows = 2 * c.Hkv * c.L;
  uint4 x[kWriteEach];
  uint4* to[kWriteEach];
#pragma unroll
  for (int e = 0; e < kWriteEach; ++e) {
    const int64_t p = ((int64_t)blockIdx.x * kWriteEach + e) * kWriteThreads + threadIdx.x;
    const int row = (int)min(p / U, (int64_t)rows), piece = (int)(p % U);
    to[e] = nullptr;
    if (row >= rows) continue;
    const int i = row % c.L, which = row / c.L / c.Hkv, h = row / c.L % c.Hkv;
    const int64_t pos = (int64_t)n - c.L + i;
    if (i < c.L - count || pos < 0 || pos >= len) continue;
    const int page = cache_page(c, b, (int)pos, kKidPagedWrite);
    if (page < 0) continue;
    x[e] = reinterpret_cast<const uint4*>(row_ptr<uint16_t>(which ? c.v : c.k, which ? c.lv : c.lk, b, h, i))[piece];
    to[e] = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(c.data) + paged_row(c, page, which, h, (int)pos % c.page_size)) + piece;
  }
#pragma unroll
  for (int e = 0; e < kWriteEach; ++e)
    if (to[e]) *to[e] = x[e];
}

template <int D>
cudaError_t write_d(const CacheArgs& c, cudaStream_t s) {
  const int64_t pieces = (int64_t)2 * c.Hkv * c.L * (D / 8), each = kWriteThreads * kWriteEach;
  paged_write_kernel<D><<<dim3((unsigned)((pieces + each - 1) / each), c.B), kWriteThreads, 0, s>>>(c);
  return cudaGetLastError();
}

// ---- select

// Weights as numbers that compare as they do: NaN below all, the last `recent` tokens above all.
__device__ __forceinline__ uint32_t rank_key(float w, bool recent) {
  if (recent) return 0xffffffffu;
  if (w != w) return 0u;
  const uint32_t x = __float_as_uint(w + 0.f);  // -0 becomes +0
  return x & 0x80000000u ? ~x : x | 0x80000000u;
}

constexpr int kSelectThreads = 1024, kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;

// kEach: weights a thread holds; a row longer than the cluster holds is read in rounds.
template <int kEach>
__global__ void __launch_bounds__(kSelectThreads) paged_select_kernel(EvictArgs a) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t scan[kSelectWarps][2];
  __shared__ uint32_t found[2];
  __shared__ uint32_t totals[2];
  const cg::cluster_group cluster = cg::this_cluster();
  const int cl = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const CacheArgs& c = a.c;
  const int h = blockIdx.y, b = blockIdx.z;
  const int n = cache_len(c, b, min(c.pages_per_seq * c.page_size, a.slots), kKidPagedEvict);
  const float* weights = a.weights + b * a.w_batch + h * a.w_head;
  float* out = a.new_weights + b * a.nw_batch + h * a.nw_head;
  int* kept = a.kept + ((int64_t)b * c.Hkv + h) * a.budget;
  const int stay = min(n, a.budget), old = n - a.recent;
  constexpr int kBlock = kSelectThreads * kEach;
  const int round = cl * kBlock;
  const int rounds = (n + round - 1) / round;
  // Element e of this thread in a round; a warp's elements lie side by side.
  const int mine = me * kBlock + warp * 32 * kEach + lane;
  float w[kEach];
  auto load = [&](int r) {
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int64_t j = (int64_t)r * round + mine + 32 * e;
      w[e] = j < n ? weights[j] : 0.f;
    }
  };
  load(0);

  // ---- the key of the last token that stays, and how many of those that share it do
  uint32_t limit = 0, need = 0;
  const bool all = n <= a.budget;
  if (!all) {
    uint32_t left = stay;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int x = threadIdx.x; x < kBins; x += kSelectThreads) hist[x] = 0;
      __syncthreads();
      for (int r = 0; r < rounds; ++r) {
        if (rounds > 1) load(r);
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const int64_t j = (int64_t)r * round + mine + 32 * e;
          const uint32_t key = rank_key(w[e], j >= old);
          if (j < n && (pass == 0 || key >> (shift + bits) == limit >> (shift + bits))) atomicAdd(&hist[key >> shift & ((1u << bits) - 1)], 1u);
        }
      }
      cluster.sync();
      // Bins from the largest down: two a thread.
      uint32_t mine2[2] = {0, 0};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int bin = kBins - 1 - (2 * (int)threadIdx.x + x);
        for (int p = 0; p < cl; ++p) mine2[x] += cluster.map_shared_rank(hist, p)[bin];
      }
      uint32_t sum = mine2[0] + mine2[1];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += y;
      }
      if (lane == 31) scan[warp][0] = sum;
      __syncthreads();
      uint32_t before = sum - mine2[0] - mine2[1];
      for (int x = 0; x < warp; ++x) before += scan[x][0];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (before < left && before + mine2[x] >= left) {
          found[0] = kBins - 1 - (2 * threadIdx.x + x);
          found[1] = left - before;
        }
        before += mine2[x];
      }
      cluster.sync();  // every block has read the histograms, and found is written
      limit |= found[0] << shift;
      left = found[1];
    }
    need = left;
  }

  // ---- places: every token's rank among those that stay
  uint32_t base_over = 0, base_same = 0;  // tokens of earlier rounds over the limit, and at it
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) load(r);
    uint32_t over[kEach], same[kEach], n_over = 0, n_same = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int64_t j = (int64_t)r * round + mine + 32 * e;
      const uint32_t key = rank_key(w[e], j >= old);
      over[e] = __ballot_sync(0xffffffffu, j < n && (all || key > limit));
      same[e] = __ballot_sync(0xffffffffu, j < n && !all && key == limit);
      n_over += __popc(over[e]);
      n_same += __popc(same[e]);
    }
    if (lane == 0) {
      scan[warp][0] = n_over;
      scan[warp][1] = n_same;
    }
    __syncthreads();
    uint32_t p_over = base_over, p_same = base_same;
    if (warp == 0) {
      uint32_t x = scan[lane][0], y = scan[lane][1];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, off);
        y += __shfl_xor_sync(0xffffffffu, y, off);
      }
      if (lane == 0) {
        totals[0] = x;
        totals[1] = y;
      }
    }
    for (int x = 0; x < warp; ++x) {
      p_over += scan[x][0];
      p_same += scan[x][1];
    }
    // Every block's counts; and every weight of this round has been read, so that in place the
    // stores below reach no weight that is still needed.
    cluster.sync();
    for (int p = 0; p < cl; ++p) {
      const uint32_t* y = cluster.map_shared_rank(totals, p);
      const uint32_t y0 = y[0], y1 = y[1];
      base_over += y0;
      base_same += y1;
      if (p < me) {
        p_over += y0;
        p_same += y1;
      }
    }
    const uint32_t below = (1u << lane) - 1;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const uint32_t s = p_same + __popc(same[e] & below);
      const uint32_t place = p_over + __popc(over[e] & below) + min(s, need);
      if (over[e] >> lane & 1u || (same[e] >> lane & 1u && s < need)) {
        kept[place] = r * round + mine + 32 * e;
        out[place] = w[e];
      }
      p_over += __popc(over[e]);
      p_same += __popc(same[e]);
    }
    cluster.sync();  // totals and scan are free again
  }
  // What lies behind the tokens that stay.
  for (int64_t x = stay + (int64_t)me * kSelectThreads + threadIdx.x; x < a.slots; x += (int64_t)cl * kSelectThreads) out[x] = 0.f;
  for (int64_t x = stay + (int64_t)me * kSelectThreads + threadIdx.x; x < a.budget; x += (int64_t)cl * kSelectThreads) kept[x] = -1;
}

// ---- move

constexpr int kMoveThreads = 256, kMoveEach = 8;

// Grid: (slices of a row, 2·Hkv, B); `threads` threads a slice of 16·threads bytes.
__global__ void __launch_bounds__(kMoveThreads) paged_move_kernel(EvictArgs a, int threads) {
  const CacheArgs& c = a.c;
  const int which = blockIdx.y / c.Hkv, h = blockIdx.y % c.Hkv, b = blockIdx.z;
  const int* kept = a.kept + ((int64_t)b * c.Hkv + h) * a.budget;
  const int per = kMoveThreads / threads, row = threadIdx.x / threads;
  const int piece = blockIdx.x * threads + threadIdx.x % threads;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    const int n = c.lens[b];
    a.new_lens[b] = max(0, min(min(n, min(c.pages_per_seq * c.page_size, a.slots)), a.budget));
  }
  for (int r0 = 0; r0 < a.budget; r0 += per * kMoveEach) {
    uint4 x[kMoveEach];
    uint4* to[kMoveEach];
    bool end = false;
#pragma unroll
    for (int e = 0; e < kMoveEach; ++e) {
      const int r = r0 + e * per + row;
      const int from = row < per && r < a.budget ? kept[r] : -1;
      to[e] = nullptr;
      end |= from < 0;
      if (from > r) {
        const int p0 = cache_page(c, b, from, kKidPagedEvict), p1 = cache_page(c, b, r, kKidPagedEvict);
        if (p0 >= 0 && p1 >= 0) {
          const uint16_t* src = reinterpret_cast<const uint16_t*>(c.data) + paged_row(c, p0, which, h, from % c.page_size);
          x[e] = reinterpret_cast<const uint4*>(src)[piece];
          to[e] = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(c.data) + paged_row(c, p1, which, h, r % c.page_size)) + piece;
        }
      }
    }
    // All loads of these rows before their stores; later rows lie past every row stored here.
    const bool last = __syncthreads_or(end);
#pragma unroll
    for (int e = 0; e < kMoveEach; ++e)
      if (to[e]) *to[e] = x[e];
    if (last && kept[min(r0 + per * kMoveEach, a.budget) - 1] < 0) break;
  }
}

}  // namespace

cudaError_t launch_paged_write(const CacheArgs& c, cudaStream_t s) {
  switch (c.D) {
    case 32: return write_d<32>(c, s);
    case 64: return write_d<64>(c, s);
    case 96: return write_d<96>(c, s);
    case 128: return write_d<128>(c, s);
    case 256: return write_d<256>(c, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_paged_select(const EvictArgs& a, cudaStream_t s) {
  const int64_t n = min(a.c.pages_per_seq * a.c.page_size, a.slots);
  const int each = n <= 4 * kSelectThreads ? 4 : 16;
  int cl = 1;
  while (cl < 8 && (int64_t)cl * each * kSelectThreads < n) cl *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cl, a.c.Hkv, a.c.B);
  cfg.blockDim = dim3(kSelectThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cl;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return each == 4 ? cudaLaunchKernelEx(&cfg, paged_select_kernel<4>, a) : cudaLaunchKernelEx(&cfg, paged_select_kernel<16>, a);
}

cudaError_t launch_paged_move(const EvictArgs& a, cudaStream_t s) {
  const int pieces = a.c.D / 8;  // 16-byte pieces of a row
  const int64_t rows = (int64_t)2 * a.c.Hkv * a.c.B;
  int threads = pieces;
  while (threads % 2 == 0 && threads > 2 && rows * (pieces / threads) < 4 * (int64_t)a.c.num_sms) threads /= 2;
  paged_move_kernel<<<dim3(pieces / threads, 2 * a.c.Hkv, a.c.B), kMoveThreads, 0, s>>>(a, threads);
  return cudaGetLastError();
}

}  // namespace sdpa
