// Attention over a 16-bit paged cache for few query rows a KV head, and the kernel that joins the
// chunks of a sequence (conventions in include/sdpa.h).
//
// Rows.  The G·L query rows of a KV head (row r = query r / G of head r % G of the group), at most 32 (16 at
// D = 256), are one or two tiles of 16.  A block takes them and one chunk of the sequence.  It has
// several rings, which take units of 16 tokens of that chunk in turn, and a warp a ring and row
// tile, each with a running maximum, sum and output of its own, merged at the end.  Chunks are
// joined by a second kernel, placed while the first still runs.
//
// Bound: the bytes of the cache, 4·D a token and KV head, each read once.  So a unit's keys and
// values come by bulk tensor loads into a ring, a few units ahead, without a block
// barrier (16 tokens never cross a page, whose size is a multiple of 16); the products are warp-level
// MMAs, m16n8k16, S = Q·K^T and O += P·V, whose accumulator of the first is the operand of the second.
// P enters O as two 16-bit numbers, head and remainder, so that O is as exact as with fp32 weights (in fp16
// down to what paged.h says of small ones): the second MMA is hidden behind the copies.
// The base of a row's exponents moves only when its scores have left it far behind: one vote a unit, no shuffles.
// An output that is NaN without a reason in its row's scores has met a value that is not finite,
// perhaps one that its row does not see: mend_columns looks.
//
// Two row tiles (17 to 32 rows) are two warps on one ring, with the queries' fragments in shared memory so
// that a thread has 128 registers: one warp with both tiles took 255 registers and as long (8 queries of
// 4 sequences of 8192 tokens 39 us, of 4 queries 30), and leaves fewer warps an SM.
//
// Measured (bf16, 32 query and 8 KV heads, D = 128, calls replayed from a graph): 32 sequences of 256 to
// 8192 tokens 90.8 us, 554 MB, 6.0 TB/s with the join; one of 131072 tokens 91 us, 5.9 TB/s; 200 tokens,
// D = 64, in fp16 4.9 us.  Blocks of 8 rings, one an SM, took 94.5 us for the batch, of 4 rings, two an SM, 91 to 94.
// The weights of the batch, keys alone, 48.5 us, 5.9 TB/s: blocks of 4 warps with rings of 3 units, four an
// SM (8 warps 68 us, rings of 4 55), what a token's weight was being read a unit ahead (97 us without).
#include "paged.h"

namespace sdpa {
namespace {

using tc::ex2;

// RT: row tiles of 16 rows, a warp each for every ring; kSlots: rings of a block.
template <int D, int RT, int kSlots>
struct Cfg {
  static constexpr int kCB = (D + 63) / 64;        // 64-element blocks of a row
  static constexpr int kBlk = kTile * 128;         // bytes of one block of a unit's keys or values
  static constexpr int kHalf = kCB * kBlk, kUnit = 2 * kHalf;
  static constexpr int kWarps = RT * kSlots;
  static constexpr int kStages = 3;
  static constexpr int kBlocks = kSlots == 4 && D <= 128 ? 2 : 1;  // an SM
  static constexpr int kRows = kTile * RT;
  static constexpr int kRing = kSlots * kStages * kUnit;
  static constexpr int kMerge = kWarps * kTile * (D + 4) * 4;  // every warp's output
  static constexpr bool kQSmem = RT > 1;                       // query fragments in shared memory: 128 registers a thread
  static constexpr int kQ = kRing > kMerge ? kRing : kMerge;
  static constexpr int kSmem = kQ + (kQSmem ? RT * (D / 16) * 512 : 0) + 1024;
};

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// A ring of units of 16 tokens of one KV head, keys and (kBoth) values, loaded ahead; slot `slot` of kSlots.
// Every warp that reads it follows its state; the lead one loads.
template <int D, int kSlots, int kStages, bool kBoth>
struct Ring {
  static constexpr int kCB = (D + 63) / 64, kBlk = kTile * 128, kHalf = kCB * kBlk;
  static constexpr int kUnit = kBoth ? 2 * kHalf : kHalf;
  const CUtensorMap* map;
  const CacheArgs* c;
  const int* table;
  uint8_t* base;
  uint64_t* full;
  int h, start, end, slot, lane, units;  // units: of this ring
  bool lead;
  int issued, entry, base_unit;          // entry: page of unit base_unit + lane
  uint32_t there, phase;                 // stages that hold a unit; the parity to wait for

  __device__ __forceinline__ int pos(int u) const { return start + (slot + u * kSlots) * kTile; }
  // Takes the page table's entry for unit u0 + lane, if there is such a unit and it is a page.
  __device__ __forceinline__ void take(int u0, int found, unsigned kid) {
    base_unit = u0;
    entry = -1;
    if (u0 + lane < units) {
      if ((unsigned)found < (unsigned)c->num_pages) entry = found;
      else report_error(c->err, kDevErrIndex, kid);
    }
  }
  __device__ __forceinline__ void look(int u0, unsigned kid) { take(u0, u0 + lane < units ? table[pos(u0 + lane) / c->page_size] : -1, kid); }
  // Starts the loads of the next unit (all lanes).
  __device__ __forceinline__ void issue(unsigned kid) {
    const int u = issued++, s = u % kStages;
    there &= ~(1u << s);
    if (u >= units) return;
    if (u - base_unit >= 32) look(u, kid);
    const int page = __shfl_sync(0xffffffffu, entry, u - base_unit);
    if (page < 0) return;
    there |= 1u << s;
    if (!lead) return;
    if (lane == 0) tc::mbar_arrive_expect_tx(&full[s], kUnit);
    __syncwarp();
    if (lane < kUnit / kBlk) {
      const int which = lane / kCB, cb = lane % kCB;
      tc::tma_load_4d(base + s * kUnit + lane * kBlk, map, &full[s], cb * 64, pos(u) % c->page_size, which * c->Hkv + h, page);
    }
  }
  // Waits for unit u; false if it is not there (its page is bad) or the wait gave up (ok = false).
  __device__ __forceinline__ bool wait(int u, bool& ok, const tc::WaitCtx& wc) {
    const int s = u % kStages;
    if (!(there >> s & 1u)) return false;
    ok = __all_sync(0xffffffffu, tc::mbar_wait(&full[s], phase >> s & 1u, wc));
    if (ok) phase ^= 1u << s;
    return ok;
  }
  // Lets loads still in flight land (after a wait that gave up): of every stage, its last.
  __device__ __forceinline__ void drain() {
    for (int s = 0; s < kStages; ++s) {
      if (!(there >> s & 1u)) continue;
      const uint64_t t0 = tc::globaltimer();
      while (!tc::mbar_try_wait(&full[s], phase >> s & 1u) && tc::globaltimer() - t0 < 100000000ull) {
      }
    }
  }
};

template <typename T, int D, int RT, int kSlots>
__global__ void __launch_bounds__(Cfg<D, RT, kSlots>::kWarps * 32, Cfg<D, RT, kSlots>::kBlocks)
    paged_few_kernel(const __grid_constant__ CUtensorMap map, PagedArgs a, Cut cut) {
  using C = Cfg<D, RT, kSlots>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kSlots][C::kStages];
  __shared__ float stat[kSlots][C::kRows][2];
  __shared__ int abort_flag;
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int slot = warp / RT, rt = warp % RT;  // the warps of a ring lie side by side
  const int b = blockIdx.z, h = blockIdx.y, R = a.G * c.L;
  // The page table's entries of the first units are on their way while the length is; it says which count.
  const int* table = c.pages + b * c.pages_stride;
  const int64_t guess = ((int64_t)blockIdx.x * cut.chunk + (slot + lane * kSlots) * kTile) / c.page_size;
  const int found = guess < c.pages_per_seq ? table[guess] : -1;
  const Rows rows = rows_of(c, b, a.causal, a.max_len, kKidPagedAttn);
  const int least = rows.limit(rows.first), most = rows.first < c.L ? rows.limit(c.L - 1) : 0;
  const int start = (int)min((int64_t)blockIdx.x * cut.chunk, (int64_t)most), end = (int)min((int64_t)start + cut.chunk, (int64_t)most);
  if (start >= end && cut.splits > 1) {
    asm volatile("griddepcontrol.launch_dependents;");
    return;
  }
  if (rt == 0 && lane < C::kStages) {
    tc::mbar_init(&full[slot][lane], 1);
    tc::fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    abort_flag = 0;
    tc::prefetch_tmap(&map);
  }
  __syncthreads();
  const tc::WaitCtx wc{&abort_flag, 0, a.wait_limit_ns, c.err, kKidPagedAttn};
  const int all = (end - start + kTile - 1) / kTile;
  Ring<D, kSlots, C::kStages, true> ring{&map, &c, table, smem + slot * C::kStages * C::kUnit, full[slot], h, start, end,
                                         slot, lane, all > slot ? (all - slot + kSlots - 1) / kSlots : 0, rt == 0, 0, -1, 0, 0u, 0u};
  ring.take(0, found, kKidPagedAttn);
#pragma unroll
  for (int s = 0; s < C::kStages; ++s) ring.issue(kKidPagedAttn);

  // Query rows as MMA operands; rows that are not there are zeros.
  uint32_t qa[C::kQSmem ? 1 : D / 16][4];
  uint4* const q_frag = reinterpret_cast<uint4*>(smem + C::kQ) + rt * (D / 16) * 32 + lane;  // [D / 16][lane]
  int lim[2];
  {
    const T* q[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = kTile * rt + 8 * x + g, i = r / a.G;
      lim[x] = r < R ? rows.limit(i) : 0;
      q[x] = r < R && i >= rows.first ? row_ptr<T>(a.q, a.lq, b, h * a.G + r % a.G, i) + 2 * t : nullptr;
    }
    if (!C::kQSmem || slot == 0) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = q[e % 2] ? *reinterpret_cast<const uint32_t*>(q[e % 2] + 16 * ks + 8 * (e / 2)) : 0u;
        if constexpr (C::kQSmem) {
          q_frag[ks * 32] = make_uint4(f[0], f[1], f[2], f[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) qa[ks][e] = f[e];
        }
      }
    }
    if constexpr (C::kQSmem) __syncthreads();
  }

  float o[D / 8][4], m[2] = {minus_inf(), minus_inf()}, l[2] = {0.f, 0.f};  // m: the rows' bases (paged.h)
#pragma unroll
  for (int d = 0; d < D / 8; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
  const float c2 = a.scale_log2;
  // ldmatrix rows: keys for S (matrices: keys 0-7 and 8-15, each two 8-element pieces), keys for O.
  const int k_row = lane / 16 * 8 + lane % 8, k_piece = lane / 8 % 2, v_row = lane % 16, v_piece = lane / 16;
  bool ok = true;
  for (int u = 0; u < ring.units; ++u) {
    if (ring.wait(u, ok, wc)) {
      uint8_t* unit = ring.base + u % C::kStages * C::kUnit;
      const uint32_t ks0 = tc::smem_u32(unit), vs0 = ks0 + C::kHalf;
      const int k0 = ring.pos(u);
      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t kb[4], f[4];
        ldsm(kb, ks0 + ks / 4 * C::kBlk + tc::sw128_off(k_row, ks % 4 * 2 + k_piece));
        if constexpr (C::kQSmem) {
          const uint4 x = q_frag[ks * 32];
          f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = qa[ks][e];
        }
        mma<T>(s[0], f, kb[0], kb[1]);
        mma<T>(s[1], f, kb[2], kb[3]);
      }
      // A unit that some row sees only in part: hidden scores are -inf; values that no row sees
      // become 0, since what lies there may be anything.
      const bool cut_unit = k0 + kTile > least;
      if (k0 + kTile > most) {
        for (int x = lane; x < kTile * C::kCB * 8; x += 32) {
          const int row = x / (C::kCB * 8), piece = x % (C::kCB * 8);
          if (k0 + row >= most) *reinterpret_cast<uint4*>(unit + C::kHalf + piece / 8 * C::kBlk + tc::sw128_off(row, piece % 8)) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_async_smem();  // before the stage's next load
        __syncwarp();
      }
      float top[2];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = s[n][e] * c2;
          if (cut_unit && k0 + 8 * n + 2 * t + e % 2 >= lim[e / 2]) v = minus_inf();
          s[n][e] = v;
        }
#pragma unroll
      for (int x = 0; x < 2; ++x) top[x] = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]), fmaxf(s[1][2 * x], s[1][2 * x + 1]));
      const bool rise = top[0] > base_high<T>(m[0]) || top[1] > base_high<T>(m[1]);
      const bool fall = kNarrow<T> && (top[0] < m[0] - kFall || top[1] < m[1] - kFall);  // (by the lane's scores)
      if (__any_sync(0xffffffffu, rise || fall)) {
        const bool falls = kNarrow<T> && __any_sync(0xffffffffu, fall);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float v = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
          float up = fmaxf(m[x], base_of<T>(v));
          if (falls) {
            float sum = l[x] + __shfl_xor_sync(0xffffffffu, l[x], 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (base_falls(m[x], v, sum)) up = base_of<T>(v);
          }
          const float f = up == minus_inf() ? 1.f : ex2(m[x] - up);
          m[x] = up;
          l[x] *= f;
#pragma unroll
          for (int d = 0; d < D / 8; ++d) {
            o[d][2 * x] *= f;
            o[d][2 * x + 1] *= f;
          }
        }
      }
      uint32_t hi[4], lo[4];  // P and what its rounding leaves, as operands
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float shift = m[x] == minus_inf() ? 0.f : m[x];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = ex2(s[n][2 * x] - shift), p1 = ex2(s[n][2 * x + 1] - shift);
          l[x] += p0 + p1;
          const uint32_t w = tc::pack2<T>(p0, p1);
          float h0, h1;
          tc::unpack2<T>(w, h0, h1);
          hi[2 * n + x] = w;
          lo[2 * n + x] = tc::pack2<T>(p0 - h0, p1 - h1);
        }
      }
#pragma unroll
      for (int dd = 0; dd < D / 16; ++dd) {
        uint32_t vb[4];
        ldsm_t(vb, vs0 + dd / 4 * C::kBlk + tc::sw128_off(v_row, dd % 4 * 2 + v_piece));
        mma<T>(o[2 * dd], hi, vb[0], vb[1]);
        mma<T>(o[2 * dd + 1], hi, vb[2], vb[3]);
        mma<T>(o[2 * dd], lo, vb[0], vb[1]);
        mma<T>(o[2 * dd + 1], lo, vb[2], vb[3]);
      }
    }
    // The ring's warps are done with the unit; all of them go on, or none.
    if constexpr (RT > 1) ok = tc::named_sync_and(1 + slot, 32 * RT, ok);
    else __syncwarp();
    if (!ok) break;
    ring.issue(kKidPagedAttn);
  }
  if (!ok) ring.drain();

  // ---- the warps' results
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    if (lim[x] == 0) {  // a row that sees nothing
      m[x] = minus_inf();
      l[x] = 0.f;
    }
    if (t == 0) {
      stat[slot][kTile * rt + 8 * x + g][0] = m[x];
      stat[slot][kTile * rt + 8 * x + g][1] = l[x];
    }
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;");
  float* red = reinterpret_cast<float*>(smem);  // [slot][row][D + 4]
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int q = kTile * rt + 8 * x + g;
    float M = minus_inf();
#pragma unroll
    for (int w = 0; w < kSlots; ++w) M = fmaxf(M, stat[w][q][0]);
    // (a warp that saw nothing but NaN has no maximum and a sum of NaN)
    const float wgt = m[x] == minus_inf() ? 1.f : ex2(m[x] - M);
    float* to = red + (slot * C::kRows + q) * (D + 4) + 2 * t;
#pragma unroll
    for (int d = 0; d < D / 8; ++d)
      *reinterpret_cast<float2*>(to + 8 * d) = lim[x] == 0 ? make_float2(0.f, 0.f) : make_float2(o[d][2 * x] * wgt, o[d][2 * x + 1] * wgt);
  }
  __syncthreads();
  for (int y = threadIdx.x; y < C::kRows * (D / 4); y += C::kWarps * 32) {
    const int q = y / (D / 4), d = y % (D / 4) * 4;
    if (q >= R) continue;
    float M = minus_inf(), sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kSlots; ++w) M = fmaxf(M, stat[w][q][0]);
#pragma unroll
    for (int w = 0; w < kSlots; ++w) {
      const float mw = stat[w][q][0], lw = stat[w][q][1];
      sum += mw == minus_inf() ? lw : lw * ex2(mw - M);
      const float4 z = *reinterpret_cast<const float4*>(red + (w * C::kRows + q) * (D + 4) + d);
      v.x += z.x; v.y += z.y; v.z += z.z; v.w += z.w;
    }
    const int hq = h * a.G + q % a.G, i = q / a.G;
    const int64_t row = ((int64_t)b * a.Hq + hq) * c.L + i;
    if (sum == sum && (v.x != v.x || v.y != v.y || v.z != v.z || v.w != v.w)) {
      float x[4] = {v.x, v.y, v.z, v.w};
      if (sum > 0.f) mend_columns<T, D, 4>(a, b, h, hq, i, d, start, min(end, rows.limit(i)), M, x);
      else x[0] = x[1] = x[2] = x[3] = 0.f;  // nothing seen but scores of -inf
      v = make_float4(x[0], x[1], x[2], x[3]);
    }
    if (cut.splits > 1) {
      const int64_t at = part_of(cut, b, a.Hq, hq, i, blockIdx.x);
      *reinterpret_cast<float4*>(a.workspace + at * D + d) = v;
      if (d == 0) {
        float* ml = part_stats(a, cut) + 2 * at;
        ml[0] = M;
        ml[1] = sum;
      }
    } else {
      const float fold = fold_sink(a.sinks, hq, M, sum), inv = sum == 0.f ? 0.f : fold / sum;
      T* out = row_ptr<T>(a.out, a.lo, b, hq, i) + d;
      *reinterpret_cast<uint2*>(out) = make_uint2(tc::pack2<T>(v.x * inv, v.y * inv), tc::pack2<T>(v.z * inv, v.w * inv));
      if (a.lse && d == 0) a.lse[row] = sum == 0.f ? minus_inf() : (M + log2f(sum)) * kLn2;
    }
  }
}

// Joins the chunks of a query row, kWarps warps a row, each the chunks x, x + kWarps, ...; 8 warps a block.
constexpr int kJoinWarps = 8;
template <typename T, int D, int kWarps>
__global__ void __launch_bounds__(32 * kJoinWarps) paged_join_kernel(PagedArgs a, Cut cut) {
  constexpr int U = D / 4, kMine = (U + 31) / 32;  // float4s of a row, and of a lane
  __shared__ float4 part[kWarps > 1 ? kJoinWarps : 1][U];
  __shared__ float stat[kWarps > 1 ? kJoinWarps : 1][2];
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, side = warp % kWarps;
  const int64_t row = (int64_t)blockIdx.x * (kJoinWarps / kWarps) + warp / kWarps;
  const bool there = row < (int64_t)c.B * a.Hq * cut.rows;
  const int i = (int)(row % cut.rows), hq = (int)(row / cut.rows % a.Hq), b = (int)(row / cut.rows / a.Hq);
  int n = 0;  // chunks that the row sees
  if (there) {
    const Rows rows = rows_of(c, b, a.causal, a.max_len, kKidPagedAttn);
    n = (int)(((int64_t)rows.limit(i) + cut.chunk - 1) / cut.chunk);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (kWarps == 1 && !there) return;
  const float* ml = part_stats(a, cut) + 2 * row * cut.splits;
  const float* from = a.workspace + row * cut.splits * D;
  float M = minus_inf(), L = 0.f;
  for (int x = lane; x < n; x += 32) M = fmaxf(M, ml[2 * x]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float4 v[kMine];
#pragma unroll
  for (int u = 0; u < kMine; ++u) v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int x = side; x < n; x += kWarps) {
    // (a chunk without a maximum has a sum of 0, or NaN and outputs of NaN)
    const float mx = ml[2 * x], w = mx == minus_inf() ? 1.f : tc::ex2(mx - M);
    L = fmaf(w, ml[2 * x + 1], L);
#pragma unroll
    for (int u = 0; u < kMine; ++u)
      if (u * 32 + lane < U) {
        const float4 y = reinterpret_cast<const float4*>(from + (int64_t)x * D)[u * 32 + lane];
        v[u].x = fmaf(w, y.x, v[u].x);
        v[u].y = fmaf(w, y.y, v[u].y);
        v[u].z = fmaf(w, y.z, v[u].z);
        v[u].w = fmaf(w, y.w, v[u].w);
      }
  }
  if constexpr (kWarps > 1) {
#pragma unroll
    for (int u = 0; u < kMine; ++u)
      if (u * 32 + lane < U) part[warp][u * 32 + lane] = v[u];
    if (lane == 0) stat[warp][0] = L;
    __syncthreads();
    if (side > 0 || !there) return;
#pragma unroll
    for (int y = 1; y < kWarps; ++y) {
      L += stat[warp + y][0];
#pragma unroll
      for (int u = 0; u < kMine; ++u)
        if (u * 32 + lane < U) {
          const float4 z = part[warp + y][u * 32 + lane];
          v[u].x += z.x; v[u].y += z.y; v[u].z += z.z; v[u].w += z.w;
        }
    }
  }
  const float fold = fold_sink(a.sinks, hq, M, L), inv = L == 0.f ? 0.f : fold / L;
  T* out = row_ptr<T>(a.out, a.lo, b, hq, i);
#pragma unroll
  for (int u = 0; u < kMine; ++u)
    if (u * 32 + lane < U)
      *reinterpret_cast<uint2*>(out + 4 * (u * 32 + lane)) = make_uint2(tc::pack2<T>(v[u].x * inv, v[u].y * inv), tc::pack2<T>(v[u].z * inv, v[u].w * inv));
  if (a.lse && lane == 0) a.lse[((int64_t)b * a.Hq + hq) * c.L + i] = L == 0.f ? minus_inf() : (M + log2f(L)) * kLn2;
}

// ---- the weights of few rows.  A warp owns its units' tokens, so sums have one order and no atomics.
template <int D, int NT>
struct WCfg {
  static constexpr int kNT = NT, kRows = kTile * kNT;
  static constexpr int kWarps = 4, kStages = 3;
  static constexpr int kUnit = (D + 63) / 64 * kTile * 128;
  static constexpr int kSmem = kWarps * kStages * kUnit + 1024;
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(WCfg<D, NT>::kWarps * 32) paged_weights_kernel(const __grid_constant__ CUtensorMap map, PagedArgs a, int chunk) {
  using C = WCfg<D, NT>;
  constexpr int kWarps = C::kWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kWarps][C::kStages];
  __shared__ int abort_flag;
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int b = blockIdx.z, h = blockIdx.y;
  const Rows rows = rows_of(c, b, a.causal, a.max_len, kKidPagedWeights);
  if (rows.first >= c.L) return;  // no real row
  const int R = a.G * c.L, start = blockIdx.x * chunk;
  if (start >= rows.len) return;
  if (lane < C::kStages) {
    tc::mbar_init(&full[warp][lane], 1);
    tc::fence_mbar_init();
  }
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();
  const tc::WaitCtx wc{&abort_flag, 0, a.wait_limit_ns, c.err, kKidPagedWeights};
  const int fresh = rows.len - (c.L - rows.first);  // tokens from here on are the call's own
  float* weights = a.weights + b * a.w_batch + h * a.w_head;
  uint32_t phase = 0;
  bool ok = true;
  // From the last rows, which see every token, to the first real ones.
  for (int row0 = (R - 1) / C::kRows * C::kRows; ok && row0 >= 0 && (min(R, row0 + C::kRows) - 1) / a.G >= rows.first; row0 -= C::kRows) {
    const bool first_pass = row0 + C::kRows >= R;
    const int i_last = (min(R, row0 + C::kRows) - 1) / a.G;
    const int end = min(start + chunk, first_pass ? rows.len : rows.limit(i_last));
    const int all = end > start ? (end - start + kTile - 1) / kTile : 0;
    Ring<D, kWarps, C::kStages, false> ring{&map, &c, c.pages + b * c.pages_stride, smem + warp * C::kStages * C::kUnit, full[warp], h, start, end,
                                            warp, lane, all > warp ? (all - warp + kWarps - 1) / kWarps : 0, true, 0, -1, 0, 0u, phase};
    ring.look(0, kKidPagedWeights);
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) ring.issue(kKidPagedWeights);
    uint32_t qa[NT][D / 16][4];
    int lim[NT][2];
    float hi[NT][2], lo[NT][2];  // lse·log2(e) in two parts
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = row0 + kTile * nt + 8 * x + g, i = r / a.G;
        const bool real = r < R && i >= rows.first;
        const int hq = h * a.G + r % a.G;
        const float lse = real ? a.lse[((int64_t)b * a.Hq + hq) * c.L + i] : minus_inf();
        lim[nt][x] = real && lse != minus_inf() ? rows.limit(i) : 0;
        hi[nt][x] = lse * kLog2e;
        // (1.93e-8: log2(e) less its fp32 number)
        lo[nt][x] = fabsf(hi[nt][x]) < __builtin_huge_valf() ? fmaf(lse, kLog2e, -hi[nt][x]) + lse * 1.92596299e-8f : 0.f;
        const T* q = real ? row_ptr<T>(a.q, a.lq, b, hq, i) + 2 * t : nullptr;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int k8 = 0; k8 < 2; ++k8) qa[nt][ks][x + 2 * k8] = real ? *reinterpret_cast<const uint32_t*>(q + 16 * ks + 8 * k8) : 0u;
      }
    const int k_row = lane / 16 * 8 + lane % 8, k_piece = lane / 8 % 2;
    // Lanes of the first four g write a token's weight each; what it was is read a unit ahead.
    const int my_key = 8 * (g / 2) + 2 * t + g % 2;
    auto was = [&](int u) {
      const int key = ring.pos(u) + my_key;
      return u < ring.units && g < 4 && key < end && !(first_pass && key >= fresh) ? weights[key] : 0.f;
    };
    float old = was(0);
    for (int u = 0; u < ring.units; ++u) {
      const int k0 = ring.pos(u);
      const float next_old = was(u + 1);
      float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
      if (ring.wait(u, ok, wc)) {
        const uint32_t ks0 = tc::smem_u32(ring.base + u % C::kStages * C::kUnit);
        float s[NT][2][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][n][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t kb[4];
          ldsm(kb, ks0 + ks / 4 * (kTile * 128) + tc::sw128_off(k_row, ks % 4 * 2 + k_piece));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma<T>(s[nt][0], qa[nt][ks], kb[0], kb[1]);
            mma<T>(s[nt][1], qa[nt][ks], kb[2], kb[3]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int x = e / 2;
              const float p = ex2(fmaf(s[nt][n][e], a.scale_log2, -hi[nt][x]) - lo[nt][x]);
              sum[n][e % 2] += k0 + 8 * n + 2 * t + e % 2 < lim[nt][x] ? p : 0.f;
            }
      }
      if (!ok) {
        ring.drain();
        break;
      }
      __syncwarp();
      ring.issue(kKidPagedWeights);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int off = 4; off <= 16; off <<= 1) sum[n][e] += __shfl_xor_sync(0xffffffffu, sum[n][e], off);
      if (g < 4 && k0 + my_key < end) weights[k0 + my_key] = old + (g & 2 ? (g & 1 ? sum[1][1] : sum[1][0]) : (g & 1 ? sum[0][1] : sum[0][0]));
      old = next_old;
    }
    phase = ring.phase;
    __syncwarp();
  }
}

// ---- host

// Rows of a block, which holds all of a KV head (of the weights: of a pass).
int rows_a_block(const PagedArgs& a) { return a.c.D == 256 || a.G * a.c.L <= kTile ? kTile : 2 * kTile; }
// Rings of a block: 4, and two blocks an SM, or 8 for a sequence that one block reads alone (200 tokens,
// D = 64: 6.3 us instead of 8.3).
int slots_of(const PagedArgs& a) { return a.c.D < 256 && rows_a_block(a) == kTile && a.max_len <= 512 ? 8 : 4; }

// How a call's sequences are cut into chunks, by the longest one that the call admits (max_len, or the
// table's width; a bound far above the sequences costs: one of 2048 tokens takes 7.2 us, under a table of 131072
// without a max_len 34.5): for few pairs of a sequence and head into one wave of
// blocks, of at least 128 tokens (2048 tokens, 8 heads: 10.3 us, of 256 12.3, of 512 14.4); for many into
// chunks of 2048 at most, so that unequal sequences share the SMs (32 of 256 to 8192 tokens, 32 rows: 125 us,
// of 1024 131, of 512 162); none where one block's warps read the sequence in what a join costs.
Cut cut_few(const PagedArgs& a) {
  constexpr int kStep = 64;  // tokens: a unit a ring
  const int64_t slots = (int64_t)(a.c.num_sms > 0 ? a.c.num_sms : 1) * (a.c.D == 256 ? 1 : 2);
  const int64_t pairs = (int64_t)a.c.B * a.c.Hkv;
  const int64_t want = max((int64_t)1, slots / pairs);
  int64_t chunk = (a.max_len + want - 1) / want;
  if (pairs * 4 > slots) chunk = min(chunk, (int64_t)2048);
  chunk = a.max_len <= 512 ? a.max_len : max(chunk, (int64_t)128);
  // Partial results take at most 64 MiB.
  const int64_t partial = (int64_t)a.c.B * a.Hq * a.c.L * (a.c.D + 2) * (int64_t)sizeof(float);
  const int64_t most = max((int64_t)1, ((int64_t)64 << 20) / partial);
  chunk = max(chunk, (a.max_len + most - 1) / most);
  Cut cut;
  cut.chunk = (int)min((chunk + kStep - 1) / kStep * kStep, (int64_t)1 << 30);
  cut.splits = (a.max_len + cut.chunk - 1) / cut.chunk;
  cut.rows = a.c.L;
  return cut;
}

Cut cut_of(const PagedArgs& a) { return paged_chunk_takes(a) ? paged_chunk_cut(a) : cut_few(a); }

template <typename T, int D, int RT, int kSlots>
cudaError_t few_t(const PagedArgs& a, cudaStream_t s) {
  using C = Cfg<D, RT, kSlots>;
  auto* kern = paged_few_kernel<T, D, RT, kSlots>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(kern, C::kSmem, ready);
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  if (!make_tmap_pages(&map, a.c, kTile)) return cudaErrorInvalidValue;
  const Cut cut = cut_few(a);
  kern<<<dim3(cut.splits, a.c.Hkv, a.c.B), C::kWarps * 32, C::kSmem, s>>>(map, a, cut);
  return cudaGetLastError();
}

template <typename T, int D, int NT>
cudaError_t weights_nt(const PagedArgs& a, cudaStream_t s) {
  using C = WCfg<D, NT>;
  auto* kern = paged_weights_kernel<T, D, NT>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(kern, C::kSmem, ready);
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  if (!make_tmap_pages(&map, a.c, kTile)) return cudaErrorInvalidValue;
  const int chunk = 1024;
  kern<<<dim3((a.max_len + chunk - 1) / chunk, a.c.Hkv, a.c.B), C::kWarps * 32, C::kSmem, s>>>(map, a, chunk);
  return cudaGetLastError();
}

template <typename T, int D, int kWarps>
cudaError_t join_t(const PagedArgs& a, const Cut& cut, cudaStream_t s) {
  constexpr int kRows = kJoinWarps / kWarps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)a.c.B * a.Hq * cut.rows + kRows - 1) / kRows));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];  // its blocks may be placed while the last chunks are still running
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<T, D, kWarps>, a, cut);
}

enum class Do { kAttn, kJoin, kWeights };

template <typename T, int D>
cudaError_t run_d(const PagedArgs& a, Do what, cudaStream_t s) {
  if (what == Do::kJoin) {
    const Cut cut = cut_of(a);
    return cut.splits > 8 ? join_t<T, D, kJoinWarps>(a, cut, s) : join_t<T, D, 1>(a, cut, s);
  }
  if (what == Do::kWeights) {
    if constexpr (D == 256) return weights_nt<T, D, 1>(a, s);
    else return rows_a_block(a) == kTile ? weights_nt<T, D, 1>(a, s) : weights_nt<T, D, 2>(a, s);
  }
  if constexpr (D == 256) return few_t<T, D, 1, 4>(a, s);
  else if (rows_a_block(a) > kTile) return few_t<T, D, 2, 4>(a, s);
  else return slots_of(a) == 8 ? few_t<T, D, 1, 8>(a, s) : few_t<T, D, 1, 4>(a, s);
}

template <typename T>
cudaError_t run_t(const PagedArgs& a, Do what, cudaStream_t s) {
  switch (a.c.D) {
    case 32: return run_d<T, 32>(a, what, s);
    case 64: return run_d<T, 64>(a, what, s);
    case 96: return run_d<T, 96>(a, what, s);
    case 128: return run_d<T, 128>(a, what, s);
    case 256: return run_d<T, 256>(a, what, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t run(const PagedArgs& a, int dtype, Do what, cudaStream_t s) {
  return dtype == 1 ? run_t<__half>(a, what, s) : run_t<__nv_bfloat16>(a, what, s);
}

}  // namespace

bool paged_attn_launchable(const PagedArgs& a) { return !paged_chunk_takes(a) || paged_chunk_blocks(a) <= 0x7fffffff; }
size_t paged_attn_workspace(const PagedArgs& a) {
  const Cut cut = cut_of(a);
  return cut.splits == 1 ? 0 : (size_t)a.c.B * a.Hq * cut.rows * cut.splits * (a.c.D + 2) * sizeof(float);
}
cudaError_t launch_paged_attn(const PagedArgs& a, int dtype, cudaStream_t s) {
  return paged_chunk_takes(a) ? launch_paged_chunk(a, dtype, s) : run(a, dtype, Do::kAttn, s);
}
cudaError_t launch_paged_join(const PagedArgs& a, int dtype, cudaStream_t s) { return run(a, dtype, Do::kJoin, s); }
cudaError_t launch_paged_weights(const PagedArgs& a, int dtype, cudaStream_t s) {
  return paged_gain_takes(a) ? launch_paged_gain(a, dtype, s) : run(a, dtype, Do::kWeights, s);
}

}  // namespace sdpa
