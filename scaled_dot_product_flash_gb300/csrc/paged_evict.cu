// Writing a 16-bit paged cache, and evicting the tokens that have gathered the least attention
// weight (conventions in include/sdpa.h).
//
// Write: every thread moves four 16-byte pieces.  Bound: HBM for prompts, latency for tokens: two prompts of
// 4096 tokens, 8 heads, D = 128 8.3 us from a graph (67 MB in and out, half of it to L2), one token of 32
// sequences 2.3.
//
// Evict, two kernels:
//  - select: a cluster of blocks takes one row of weights (one sequence and KV head).  Weights are
//    ranked as 32-bit keys in their order; four histograms of 8 bits, summed over the
//    cluster through distributed shared memory, give the key of the last token that stays, and
//    counts of what lies before each token (ballots in a warp, then warps, then blocks) its new place.
//  - move: kept[r] >= r and both ascend, so a block that loads rows in order and stores them only
//    when all of its loads have landed never overwrites a row that is still to be read.  Rows are cut
//    into slices of 32 bytes or more, one block each: slices do not touch one another, and there are
//    enough of them to fill the device.
//    Bound: HBM, twice the rows that move.  32 sequences of 2304 tokens to 2048, 8 heads, D = 128: 99 us
//    with the selection (8 of them), 5.5 TB/s; looking places up a round ahead but waiting for it, 128.
//    One of 32768 to 8192: 28.6 us, 12 of them the selection, whose cluster barriers cost 0.7 us each; eight
//    rounds of 1024 rows in slices of 32 bytes.
#include <cooperative_groups.h>

#include "paged.h"

namespace sdpa {
namespace {

namespace cg = cooperative_groups;

constexpr int kWriteEach = 4;

// Grid: (blocks of rows · keys and values of each head, sequences); `per` rows are moved at a time.
template <int D>
__global__ void __launch_bounds__(256) paged_write_kernel(CacheArgs c, int per, int chunks, Divider by_page) {
  constexpr int U = D / 8;  // 16-byte pieces of a row
  const int b = blockIdx.y, head = blockIdx.x / chunks, which = head >= c.Hkv, h = head - which * c.Hkv;
  const int row = threadIdx.x / U, piece = threadIdx.x % U, i0 = (blockIdx.x - head * chunks) * per * kWriteEach + row;
  const int len = cache_len(c, b, c.pages_per_seq * c.page_size, kKidPagedWrite);
  // (a sequence whose length lies past the table's end keeps its rows' positions)
  const int64_t first = (int64_t)max(c.lens[b], 0) - c.L;
  const int pad = c.counts ? c.L - min(max(c.counts[b], 0), c.L) : 0;
  if (row >= per) return;
  const uint16_t* from = row_ptr<uint16_t>(which ? c.v : c.k, which ? c.lv : c.lk, b, h, 0) + 8 * piece;
  const int64_t stride = which ? c.lv.sl : c.lk.sl;
  const int* table = c.pages + b * c.pages_stride;
  uint4 x[kWriteEach];
  int page[kWriteEach], place[kWriteEach];
#pragma unroll
  for (int e = 0; e < kWriteEach; ++e) {
    const int i = i0 + e * per;
    const int64_t pos = first + i;
    page[e] = -1;
    if (i >= c.L || i < pad || pos < 0 || pos >= len) continue;
    const int slot = by_page((int)pos);
    page[e] = table[slot];
    place[e] = (int)pos - slot * c.page_size;
    x[e] = *reinterpret_cast<const uint4*>(from + i * stride);
  }
#pragma unroll
  for (int e = 0; e < kWriteEach; ++e) {
    if ((unsigned)page[e] < (unsigned)c.num_pages)
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(c.data) + paged_row(c, page[e], which, h, place[e]) + 8 * piece) = x[e];
    else if (i0 + e * per < c.L && i0 + e * per >= pad && first + i0 + e * per >= 0 && first + i0 + e * per < len)
      report_error(c.err, kDevErrIndex, kKidPagedWrite);
  }
}

template <int D>
cudaError_t write_d(const CacheArgs& c, cudaStream_t s) {
  const int per = min(c.L, 256 / (D / 8)), threads = (per * (D / 8) + 31) / 32 * 32;
  const int chunks = (c.L + per * kWriteEach - 1) / (per * kWriteEach);
  paged_write_kernel<D><<<dim3((unsigned)(2 * (int64_t)c.Hkv * chunks), c.B), threads, 0, s>>>(c, per, chunks, divider(c.page_size));
  return cudaGetLastError();
}

// ---- select

// Weights as numbers above 0 that compare as they do, NaN below all.
__device__ __forceinline__ uint32_t rank_key(float w) {
  if (w != w) return 1u;
  const uint32_t x = __float_as_uint(w + 0.f);  // -0 becomes +0
  return x & 0x80000000u ? ~x : x | 0x80000000u;
}

constexpr int kBins = 256, kCopies = 4, kMaxCluster = 8;

// Σ over the warps before this one, of a warp's sums that every thread passes in.
template <int kWarps>
__device__ __forceinline__ uint32_t before_warp(const uint32_t (&sums)[kWarps], int warp, int lane) {
  return __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0u);
}

// kEach: weights a thread holds; a row longer than the cluster holds is read in rounds.  The last
// `recent` tokens are not ranked: their places are known.
template <int kThreads, int kEach>
__global__ void __launch_bounds__(kThreads) paged_select_kernel(EvictArgs a) {
  constexpr int kWarps = kThreads / 32;
  static_assert(kThreads >= kBins && kEach <= 32, "a bin a thread, a bit an element");
  __shared__ uint4 hist[kBins];          // kCopies counts a bin, one for each lane mod 4: fewer lanes meet at one
  __shared__ uint32_t counts[2][kBins];  // their sums, two in turn: other blocks read one while the next is made
  __shared__ uint32_t scan[2][kWarps];
  __shared__ uint32_t found[2];
  __shared__ uint32_t totals[2], earlier[2];
  asm volatile("griddepcontrol.launch_dependents;");  // the move may take its place: it waits for this grid
  const cg::cluster_group cluster = cg::this_cluster();
  const int cl = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const CacheArgs& c = a.c;
  const int h = blockIdx.y, b = blockIdx.z;
  const int n = cache_len(c, b, min(c.pages_per_seq * c.page_size, a.slots), kKidPagedEvict);
  const float* weights = a.weights + b * a.w_batch + h * a.w_head;
  float* out = a.new_weights + b * a.nw_batch + h * a.nw_head;
  int* kept = a.kept + ((int64_t)b * c.Hkv + h) * a.budget;
  const bool all = n <= a.budget;
  const int stay = min(n, a.budget), ranked = all ? n : n - a.recent;  // tokens [0, ranked) are ranked, or all stay
  constexpr int kBlock = kThreads * kEach;
  const int round = cl * kBlock;
  const int rounds = (ranked + round - 1) / round;
  // Element e of this thread in a round lies at mine + 32·e; a warp's elements lie side by side.
  const int mine = me * kBlock + warp * 32 * kEach + lane;
  uint32_t key[kEach];  // 0: no token
  auto load = [&](int r) {
    const int64_t first = (int64_t)r * round + mine;
#pragma unroll
    for (int e = 0; e < kEach; ++e) key[e] = first + 32 * e < ranked ? __float_as_uint(weights[first + 32 * e]) : 0u;
#pragma unroll
    for (int e = 0; e < kEach; ++e) key[e] = first + 32 * e < ranked ? rank_key(__uint_as_float(key[e])) : 0u;
  };
  load(0);
  auto sync = [&] {  // of all who share the row
    if (cl > 1) cluster.sync();
    else __syncthreads();
  };

  // ---- the key of the last token that stays, and how many of those that share it do
  uint32_t limit = 0, need = 0;
  if (!all && stay > a.recent) {
    need = stay - a.recent;
    for (int shift = 24; shift >= 0; shift -= 8) {
      uint32_t* mine_too = counts[shift / 8 % 2];
      if (threadIdx.x < kBins) hist[threadIdx.x] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      for (int r = 0; r < rounds; ++r) {
        if (rounds > 1) load(r);
        uint32_t* mine_of = reinterpret_cast<uint32_t*>(hist) + lane % kCopies;
#pragma unroll
        for (int e = 0; e < kEach; ++e)
          if (key[e] && (shift == 24 || (key[e] ^ limit) >> (shift + 8) == 0)) atomicAdd(mine_of + (key[e] >> shift & 255u) * kCopies, 1u);
      }
      __syncthreads();
      if (threadIdx.x < kBins) {  // bins from the largest down, one for each of the first threads
        const uint4 y = hist[kBins - 1 - threadIdx.x];
        mine_too[threadIdx.x] = y.x + y.y + y.z + y.w;
      }
      if (cl > 1) cluster.sync();
      uint32_t own = 0, upto = 0;
      if (threadIdx.x < kBins) {
        if (cl == 1) own = mine_too[threadIdx.x];
        else {  // all of them on their way at once
#pragma unroll
          for (int p = 0; p < kMaxCluster; ++p)
            if (p < cl) own += cluster.map_shared_rank(mine_too, p)[threadIdx.x];
        }
        upto = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += y;
        }
        if (lane == 31) scan[0][warp] = upto;
      }
      __syncthreads();
      if (threadIdx.x < kBins) {
        const uint32_t before = upto - own + before_warp(scan[0], warp, lane);
        if (before < need && before + own >= need) {
          found[0] = kBins - 1 - threadIdx.x;
          found[1] = need - before;
        }
      }
      __syncthreads();
      limit |= found[0] << shift;
      need = found[1];
    }
  } else if (!all) {
    limit = 0xffffffffu;  // nothing but recent tokens stays
  }

  // ---- places: every token's rank among those that stay
  uint32_t base_over = 0, base_same = 0;  // tokens of earlier rounds over the limit, and at it
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) load(r);
    uint32_t over = 0, same = 0;  // bit e: element e is over the limit, or at it
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      over |= (key[e] > limit ? 1u : 0u) << e;
      same |= (key[e] == limit && limit ? 1u : 0u) << e;
    }
    const uint32_t n_over = __reduce_add_sync(0xffffffffu, __popc(over)), n_same = __reduce_add_sync(0xffffffffu, __popc(same));
    if (lane == 0) {
      scan[0][warp] = n_over;
      scan[1][warp] = n_same;
    }
    __syncthreads();
    uint32_t p_over = base_over + before_warp(scan[0], warp, lane), p_same = base_same + before_warp(scan[1], warp, lane);
    if (threadIdx.x == kThreads - 1) {
      totals[0] = p_over - base_over + n_over;
      totals[1] = p_same - base_same + n_same;
    }
    // The weights once more, as they are.  In place no store below reaches a weight of a later round.
    float w[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if ((over | same) >> e & 1u) w[e] = weights[(int64_t)r * round + mine + 32 * e];
    sync();  // every block's counts are there, and its weights read
    if (cl > 1) {
      if (warp == 0) {
        uint32_t y[2] = {0, 0};
        if (lane < cl) {
          const uint32_t* x = cluster.map_shared_rank(totals, lane);
          y[0] = x[0];
          y[1] = x[1];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t sum = __reduce_add_sync(0xffffffffu, y[k]), mine_first = __reduce_add_sync(0xffffffffu, lane < me ? y[k] : 0u);
          if (lane == 0) {
            found[k] = mine_first;
            earlier[k] = sum;
          }
        }
      }
      __syncthreads();
      p_over += found[0];
      p_same += found[1];
      base_over += earlier[0];
      base_same += earlier[1];
    } else {
      base_over += totals[0];
      base_same += totals[1];
    }
    const uint32_t below = (1u << lane) - 1;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const uint32_t o = __ballot_sync(0xffffffffu, over >> e & 1u), t = __ballot_sync(0xffffffffu, same >> e & 1u);
      const uint32_t nth = p_same + __popc(t & below), place = p_over + __popc(o & below) + min(nth, need);
      if (over >> e & 1u || (same >> e & 1u && nth < need)) {
        kept[place] = r * round + mine + 32 * e;
        out[place] = w[e];
      }
      p_over += __popc(o);
      p_same += __popc(t);
    }
    if (r + 1 < rounds) sync();  // totals and scan are free again
  }
  // The recent tokens, and what lies behind the kept ones.  In place a step's loads come before its
  // stores, and all of them before the zeros.
  const bool in_place = a.weights == a.new_weights;
  if (!all) {
    const int first = stay - a.recent;
    for (int x = 0; x < a.recent; x += round) {
      float w[kEach];
#pragma unroll
      for (int e = 0; e < kEach; ++e)
        if ((int64_t)x + mine + 32 * e < a.recent) w[e] = weights[ranked + x + mine + 32 * e];
      if (in_place) sync();
#pragma unroll
      for (int e = 0; e < kEach; ++e)
        if ((int64_t)x + mine + 32 * e < a.recent) {
          kept[first + x + mine + 32 * e] = ranked + x + mine + 32 * e;
          out[first + x + mine + 32 * e] = w[e];
        }
    }
    if (in_place) sync();
  }
  for (int64_t x = stay + (int64_t)me * kThreads + threadIdx.x; x < a.slots; x += (int64_t)cl * kThreads) out[x] = 0.f;
  for (int64_t x = stay + (int64_t)me * kThreads + threadIdx.x; x < a.budget; x += (int64_t)cl * kThreads) kept[x] = -1;
  if (cl > 1) cluster.sync();  // nobody leaves while its counts are read
}

// ---- move

constexpr int kMoveEach = 4, kMoveStages = 4;  // 16-byte pieces of a thread in a round, and rounds in shared memory

// Grid: (slices of a row, 2·Hkv, B); `threads` threads a row, 16 bytes each.  Rows go in rounds of
// kMoveEach·kThreads / threads through a ring in shared memory, loaded asynchronously a few rounds
// ahead; where a round's rows are and go is looked up one more round ahead, once a row.
// kLook: rows that a thread looks up, kMoveEach / threads rounded up.
template <int kThreads, int kLook>
__global__ void __launch_bounds__(kThreads) paged_move_kernel(EvictArgs a, int threads) {
  extern __shared__ uint4 ring[];  // [stages][kMoveEach][kThreads], then the rows' places
  const CacheArgs& c = a.c;
  const int which = blockIdx.y / c.Hkv, h = blockIdx.y - which * c.Hkv, b = blockIdx.z;
  const int* kept = a.kept + ((int64_t)b * c.Hkv + h) * a.budget;
  const int* table = c.pages + b * c.pages_stride;
  const int per = kThreads / threads, step = per * kMoveEach;
  const int row = threadIdx.x / threads, piece = blockIdx.x * threads + threadIdx.x - row * threads;
  uint2* places = reinterpret_cast<uint2*>(ring + kMoveStages * kMoveEach * kThreads);  // [stages][step]: from and to, rows of the cache
  uint4* const base = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(c.data) + paged_row(c, 0, which, h, 0)) + piece;
  const uint32_t page_rows = 2u * c.Hkv * c.page_size;
  const int row_pieces = c.D / 8;
  constexpr uint32_t kStays = 0xffffffffu;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    const int n = c.lens[b];
    a.new_lens[b] = max(0, min(min(n, min(c.pages_per_seq * c.page_size, a.slots)), a.budget));
  }
  const int rounds = (min(a.budget, min(c.pages_per_seq * c.page_size, a.slots)) + step - 1) / step;
  // A round's rows are looked up in three steps, an iteration apart, so that none waits for the one
  // before: their places in kept, the table's entries for them, and where they are and go (kStays for
  // those that are not moved).
  int next[kLook], from[kLook];
  unsigned p0[kLook], p1[kLook];
  auto look_kept = [&](int round) {
#pragma unroll
    for (int e = 0; e < kLook; ++e) {
      const int x = e * kThreads + threadIdx.x, r = round * step + x;
      next[e] = round < rounds && x < step && r < a.budget ? kept[r] : -1;
    }
  };
  auto look_pages = [&](int round) {
#pragma unroll
    for (int e = 0; e < kLook; ++e) {
      const int r = round * step + e * kThreads + threadIdx.x;
      from[e] = next[e];
      p0[e] = p1[e] = 0u;
      if (from[e] > r) {
        p0[e] = table[a.by_page(from[e])];
        p1[e] = table[a.by_page(r)];
      }
    }
  };
  auto look_done = [&](int round) {
    uint2* to = places + round % kMoveStages * step;
#pragma unroll
    for (int e = 0; e < kLook; ++e) {
      const int x = e * kThreads + threadIdx.x, r = round * step + x;
      if (round >= rounds || x >= step) break;
      uint2 y = make_uint2(kStays, 0u);
      if (from[e] > r) {
        if (p0[e] < (unsigned)c.num_pages && p1[e] < (unsigned)c.num_pages)
          y = make_uint2(p0[e] * page_rows + (from[e] - a.by_page(from[e]) * c.page_size), p1[e] * page_rows + (r - a.by_page(r) * c.page_size));
        else
          report_error(c.err, kDevErrIndex, kKidPagedEvict);
      }
      to[x] = y;
    }
  };
  auto load = [&](int round) {
    if (round < rounds && row < per) {
      const uint2* at = places + round % kMoveStages * step;
      uint4* to = ring + round % kMoveStages * kMoveEach * kThreads + threadIdx.x;
#pragma unroll
      for (int e = 0; e < kMoveEach; ++e) {
        const uint32_t from = at[e * per + row].x;
        if (from != kStays)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(to + e * kThreads)), "l"(base + (int64_t)from * row_pieces) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  look_kept(0);
#pragma unroll
  for (int x = 0; x < kMoveStages - 1; ++x) {
    look_pages(x);
    look_kept(x + 1);
    look_done(x);
  }
  look_pages(kMoveStages - 1);
  look_kept(kMoveStages);
  __syncthreads();
#pragma unroll
  for (int x = 0; x < kMoveStages - 2; ++x) load(x);
  for (int round = 0; round < rounds; ++round) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kMoveStages - 3) : "memory");
    // Every thread's loads of this round before any of its stores; later rounds' rows lie past every
    // row stored here.  (And the places that the next round's load reads are there, those that the
    // look below replaces no longer needed.)
    __syncthreads();
    load(round + kMoveStages - 2);
    if (row < per) {
      const uint2* at = places + round % kMoveStages * step;
      const uint4* x = ring + round % kMoveStages * kMoveEach * kThreads + threadIdx.x;
#pragma unroll
      for (int e = 0; e < kMoveEach; ++e) {
        const uint2 y = at[e * per + row];
        if (y.x != kStays) base[(int64_t)y.y * row_pieces] = x[e * kThreads];
      }
    }
    look_done(round + kMoveStages - 1);
    look_pages(round + kMoveStages);
    look_kept(round + kMoveStages + 1);
  }
}

template <int kThreads, int kLook>
cudaError_t move_t(const EvictArgs& a, int threads, int pieces, cudaStream_t s) {
  auto* kern = paged_move_kernel<kThreads, kLook>;
  constexpr int kMost = kMoveStages * kMoveEach * kThreads * 16 + kMoveStages * kLook * kThreads * 8;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(kern, kMost, ready);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pieces / threads, 2 * a.c.Hkv, a.c.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kMost;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];  // its blocks may be placed while the last rows are still selected
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, threads);
}

template <int kThreads, int kEach>
cudaError_t select_t(const EvictArgs& a, int cl, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cl, a.c.Hkv, a.c.B);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cl;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_select_kernel<kThreads, kEach>, a);
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
  if (n <= 4096) return select_t<512, 8>(a, 1, s);
  int cl = 1;
  while (cl < kMaxCluster && cl * (int64_t)4096 < n) cl *= 2;
  return cl * (int64_t)4096 >= n ? select_t<1024, 4>(a, cl, s) : select_t<1024, 16>(a, cl, s);
}

cudaError_t launch_paged_move(const EvictArgs& a, cudaStream_t s) {
  const int pieces = a.c.D / 8;  // 16-byte pieces of a row
  const int64_t rows = (int64_t)2 * a.c.Hkv * a.c.B, sms = a.c.num_sms > 0 ? a.c.num_sms : 1;
  // Slices of 64 bytes or more, until there are 8 blocks an SM; of 32 where even so half of the SMs
  // would have none.  32 sequences, 8 heads, D = 128, 2304 -> 2048 tokens: whole rows 106 us, slices of 128 bytes
  // 92, of 64 90; one sequence 131072 -> 32768: 64 bytes 79 us, 32 64; 8 sequences, 4 heads, D = 64:
  // 64 bytes 11 us, 32 19.
  int threads = pieces;
  while (threads % 4 == 0 && threads > 4 && rows * (pieces / threads) < 8 * sms) threads /= 2;
  if (threads == 4 && rows * (pieces / threads) < sms / 2) threads = 2;
  if (rows * (pieces / threads) >= 2 * sms) return threads < kMoveEach ? move_t<256, 2>(a, threads, pieces, s) : move_t<256, 1>(a, threads, pieces, s);
  return threads < kMoveEach ? move_t<512, 2>(a, threads, pieces, s) : move_t<512, 1>(a, threads, pieces, s);
}

}  // namespace sdpa
