// What the tcgen05 kernels of the 16-bit paged cache share: how query rows are put into tiles and
// keys into boxes, and the loads of both.
#pragma once

#include "paged.h"

namespace sdpa {
namespace tc {

constexpr int kBM = 128;  // rows of a Q tile
constexpr int kBN = 128;  // keys of a KV tile

// How query rows are put into tiles, and keys into boxes and chunks.
struct Tiling {
  int heads, tokens;  // of a Q tile
  int groups;         // of heads: G / heads
  int tiles;          // Q tiles of a block: 2, or 1 (head dim 256, and calls of one tile a KV head)
  int blocks;         // of a sequence's queries
  int whole;          // of those, from the last one on: not cut
  int box;            // tokens of a box of keys
  Cut cut;
};

template <typename T>
constexpr bool kIsBf16 = std::is_same<T, __nv_bfloat16>::value;

// Coordinates of the box of keys at position pos: its page (past the last one where there is none
// to read) and its place in it.
struct Box {
  int page, place;
};
// What the page table says about position pos (-1 past its end), which may be read before the length is known.
__device__ __forceinline__ Box entry_at(const CacheArgs& c, const int* table, int pos) {
  const int slot = pos / c.page_size;
  return Box{slot < c.pages_per_seq ? table[slot] : -1, pos - slot * c.page_size};
}
__device__ __forceinline__ Box box_of(const CacheArgs& c, const Box& entry, int pos, int end) {
  return pos < end && (unsigned)entry.page < (unsigned)c.num_pages ? entry : Box{c.num_pages, 0};
}
__device__ __forceinline__ Box box_at(const CacheArgs& c, const int* table, int pos, int end) {
  return pos < end ? box_of(c, entry_at(c, table, pos), pos, end) : Box{c.num_pages, 0};
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > 100000000ull) return;
}

// Clears the rows of a Q tile that its box does not fill.
template <int kCB>
__device__ __forceinline__ void clear_unused(uint8_t* tile, const Tiling& t) {
  const int used = t.heads * t.tokens, n = (kBM - used) * 8;
  for (int x = threadIdx.x; x < n * kCB; x += blockDim.x)
    *reinterpret_cast<uint4*>(tile + x / n * 16384 + used * 128 + x % n * 16) = make_uint4(0, 0, 0, 0);
}

}  // namespace tc

// The split of the heads that share a KV head into Q tiles, and the boxes of keys.
tc::Tiling paged_tiling(const PagedArgs& a);
// Map of q or out: boxes of `heads` heads of `tokens` rows.
inline bool make_tmap_rows(CUtensorMap* map, const void* base, const PagedArgs& a, const Layout& l, const tc::Tiling& t) {
  // (a single head's, row's or batch's stride means nothing, and may be more than a map takes)
  const int64_t D = a.c.D, dims[4] = {D, a.Hq, a.c.L, a.c.B}, strides[3] = {a.Hq > 1 ? l.sh : D, a.c.L > 1 ? l.sl : D, a.c.B > 1 ? l.sb : D};
  const int box[4] = {64, t.heads, t.tokens, 1};
  return make_tmap_box(map, base, dims, strides, box);
}

}  // namespace sdpa
