// Attention of a few query rows of a key/value head over the paged cache, and
// the join of results that were split over the keys (include/paged.h).
//
// The G query heads that share a key/value head and the sequence's new tokens
// form the rows of one small matrix: row r is token r / G, head r % G of the
// group.  An item is a tile of 8 or 16 rows of a sequence over all of their keys,
// so that every key and value is read from HBM once for the whole group.
//   S = Q K^T, m' = max(m, rowmax S), P = 2^(S - m'), l = l 2^(m - m') + sum P,
//   O = O 2^(m - m') + P V                         (S in log2 units, all fp32)
// (fp16: P = 2^(S - m' + 15), so that small weights stay in the type's range, off by
// half a step or 2^-40 of the largest; l and O likewise, until they are stored.)
//
// Bound: HBM (2 bytes x 2 D per key against 2 x 4 D x rows operations).  What
// counts is bytes in flight and an even share for every SM, so the keys are cut
// into groups, the groups of all items stand in one row, and each of the launch's
// warps takes the same number of them in sequence, across items: no warp ever
// waits for another.  It streams its groups through a ring of its own, 16 KB a
// stage, filled by TMA two groups ahead (page numbers one further), and keeps m, l
// and O of its rows in registers.  An item that one warp covers is written at
// once; of the others every warp leaves O, m and l in a slot -- a warp has at most
// two such items, its first and its last -- and a second kernel joins them in
// order, which makes the result independent of timing.  (Chunks of keys fixed on
// the host, a CTA each, gave 72 % of the copy bandwidth on 64 ragged contexts up
// to 8192: the last wave ran half empty.)
// Measured, bf16, 16 query and 2 key/value heads of 256, 64 sequences: contexts of
// 8192 178 us, 1.075 GB read, 6.0 TB/s (0.90 of the copy rate; tensor pipe 9 %,
// issue 18 %); ragged contexts up to 8192 110 us with the join.  With cp.async in
// place of TMA the ragged batch took 137 us, with the rows as the products' wide
// side 123.  One sequence of 1027 keys takes 13.5 us, all of it latency.
//
// With four warps an SM the time of a group is the latency of its instructions.
// So the products are transposed, S^T = K Q^T and O^T = V^T P^T by mma.sync
// (m16n8k16) with the keys and the features as the 16 rows and the tile's rows as
// the 8 columns: half of the products, of the softmax's values and of the
// accumulators of the other way round, and Q stays in registers.
// Rows of a page that lie behind the sequence's end, or whose page number is bad,
// can hold anything: their scores are masked and their values zeroed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kWarps = kRowWarps;  // of a CTA

// KG: keys of a group
template <int D>
struct RowsCfg {
  static constexpr int KG = D == 256 ? 16 : (D == 128 ? 32 : 64);
  static constexpr int ROW = 2 * D;  // bytes of a key
  static constexpr int STAGES = 3;
  static constexpr int STAGE = 2 * KG * ROW;  // keys and values of a group
  static constexpr int RING = kWarps * STAGES * STAGE;
  static constexpr int OFF_BAR = RING;  // per warp and stage
  static constexpr int SMEM = OFF_BAR + kWarps * STAGES * 8 + 1024;
  static_assert(SMEM + 1100 <= 232448, "shared memory budget");  // (the rest: static)
  // KG rows of D features in shared memory: blocks of 64 features, rows of 128
  // bytes, the 16-byte pieces of a row swizzled by the row -- the 128-byte swizzle
  // of TMA, and free of bank conflicts for ldmatrix.  Offset of piece c of row r:
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    return (c >> 3) * (KG * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  }
};

// Tensor maps over the cache's keys and values (innermost first): feature, row
// of a page, head, page; boxes of 64 features x 2^box_log2 rows (8 to KG).
struct RowsParams {
  AttnParams a;
  CUtensorMap k, v;
  int box_log2;
};
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* tm, int f, int r, int h,
                                        int pg, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(tm), "r"(f), "r"(r), "r"(h), "r"(pg), "r"(bar)
      : "memory");
}
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
__device__ __forceinline__ bool copies_wait(uint32_t bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_sleep(bar, parity))
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  return true;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
template <bool BF>
__device__ __forceinline__ uint16_t pack1(float v) {
  if constexpr (BF) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  else return __half_as_ushort(__float2half_rn(v));
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The weight of a score that is `d` above the maximum, in P's scale.  (The difference
// comes first: it is exact where it matters, and a large maximum would swallow the scale.)
template <bool BF>
__device__ __forceinline__ float weight(float d) {
  if constexpr (!BF) d += kTopWeight<BF>;
  return exp2_approx(d);
}

// the 8x8 matrix of 16-bit values whose row i the lanes 4i .. 4i+3 hold, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.69314718055994530942f;

// The items of one sequence: `items` (row tile, key/value head) pairs of
// `groups` groups of KG keys each, over the keys [lo, kv).  A sequence with rows
// has at least one group an item, so that rows without keys are written too.
struct Extent {
  int lo, first, groups, items;  // first: the first key that a row may see
};
__device__ __forceinline__ Extent extent_of(const AttnParams& p, const Seq& s, int kg, int tile) {
  Extent e;
  e.first = p.window > 0 ? max(0, window_begin(s.kv - s.nq, p.window)) : 0;
  e.lo = e.first & ~(kg - 1);  // groups do not straddle pages that hold whole ones
  e.groups = max((s.kv - e.lo + kg - 1) / kg, 1);
  e.items = (s.nq * p.G + tile - 1) / tile * p.c.heads;
  return e;
}
// warp w of W takes the groups [share(w), share(w + 1)) of U
__device__ __forceinline__ long long share_of(long long U, int W, int w) { return U * w / W; }
// ... and group u is warp owner(u)'s
__device__ __forceinline__ int owner_of(long long U, int W, long long u) {
  return (int)(((u + 1) * W - 1) / U);
}

// NB: blocks of 8 rows of a tile.  TMA: a group is copied as boxes of the pages'
// rows, a lane each; otherwise (pages that no box of 8 rows divides) by 16-byte
// copies.
template <int D, int NB, bool BF, bool TMA>
__global__ void __launch_bounds__(32 * kWarps)
    paged_rows_kernel(const __grid_constant__ RowsParams rp) {
  const AttnParams& p = rp.a;
  using C = RowsCfg<D>;
  constexpr int KG = C::KG, MB = KG / 16, TILE = 8 * NB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ long long sh_before[32 * kWarps + 1];
  __shared__ long long sh_warp[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the join may be set up while this grid runs
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- groups before each slice of `per` sequences; CTA 0 leaves the sums for
  // the join
  const int per = (p.b.N + 32 * kWarps - 1) / (32 * kWarps);
  const int n0 = threadIdx.x * per, n1 = min(n0 + per, p.b.N);
  long long mine = 0;
  for (int n = n0; n < n1; ++n) {
    const Extent e = extent_of(p, load_seq(p.b, n), KG, TILE);
    mine += (long long)e.items * e.groups;
  }
  long long inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) sh_warp[warp] = inc;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) inc += sh_warp[w];
  sh_before[threadIdx.x + 1] = inc;
  if (threadIdx.x == 0) sh_before[0] = 0;
  __syncthreads();
  const long long U = sh_before[32 * kWarps];
  if (blockIdx.x == 0) {
    long long at = inc - mine;
    for (int n = n0; n < n1; ++n) {
      p.before[n] = at;
      const Extent e = extent_of(p, load_seq(p.b, n), KG, TILE);
      at += (long long)e.items * e.groups;
    }
    if (threadIdx.x == 0) p.before[p.b.N] = U;
  }
  // (no more warps than groups: each of them then has a part of every item
  // between its first and its last)
  const int W = (int)min((long long)(gridDim.x * kWarps), U), w = blockIdx.x * kWarps + warp;
  if (w >= W) return;
  const long long u0 = share_of(U, W, w);
  const int steps = (int)(share_of(U, W, w + 1) - u0);

  // where a warp stands: group g of an item of a sequence
  struct Cursor {
    int n;
    Seq s;
    Extent e;
    const int32_t* table;
    int item, h, g;  // item = row tile * heads + h
  };
  auto enter = [&](Cursor& c) {  // the next sequence with rows, from c.n on
    for (; c.n < p.b.N; ++c.n) {
      c.s = load_seq(p.b, c.n);
      c.e = extent_of(p, c.s, KG, TILE);
      if (c.e.items > 0) break;
    }
    // (behind the last group there may be none: nothing reads it)
    c.table = p.b.table + min(c.n, p.b.N - 1) * p.b.table_stride;
  };
  auto advance = [&](Cursor& c) {
    if (++c.g < c.e.groups) return;
    c.g = 0;
    if (++c.h == p.c.heads) c.h = 0;
    if (++c.item < c.e.items) return;
    c.item = 0;
    ++c.n;
    enter(c);
  };
  Cursor use;
  {
    int lo = 0, hi = 32 * kWarps;  // sh_before[lo] <= u0 < sh_before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sh_before[mid] <= u0) lo = mid; else hi = mid;
    }
    long long left = u0 - sh_before[lo];
    use.n = lo * per;
    for (;;) {
      enter(use);
      const long long here = (long long)use.e.items * use.e.groups;
      if (left < here) break;
      left -= here;
      ++use.n;
    }
    use.item = (int)(left / use.e.groups);
    use.g = (int)(left - (long long)use.item * use.e.groups);
    use.h = use.item % p.c.heads;
  }
  Cursor get = use;  // the copies' cursor, ahead

  const uint32_t sm = smem_u32(smem);
  const uint32_t ring = sm + warp * C::STAGES * C::STAGE;
  const uint32_t bars = sm + C::OFF_BAR + warp * C::STAGES * 8;
  if (TMA) {
    if (lane < C::STAGES) mbar_init(bars + lane * 8, 1);
    fence_mbar_init();
    __syncwarp();
  }

  // ---- the ring.  TMA: lane l copies box l of a group (blocks of 64 features
  // side by side, then rows; keys, then values: at most 32).  Where a lane's copy
  // comes from; the page number is not looked at before the copies are issued, a
  // step after its load.
  constexpr int FC = D / 64;
  const int box_log2 = TMA ? rp.box_log2 : 0, per_kv = FC * (KG >> box_log2);  // boxes of the keys
  const bool is_v = lane >= per_kv;
  const int bx = (lane - (is_v ? per_kv : 0)) % FC, by = (lane - (is_v ? per_kv : 0)) / FC;
  const int my_row = by << box_log2;
  struct Source {
    int page, row, head;
    bool any;  // something to copy
  };
  auto lookup = [&](int st) -> Source {
    Source r{-1, 0, 0, false};
    if (!TMA || lane >= 2 * per_kv || st >= steps) return r;
    const int key = get.e.lo + get.g * KG + my_row;
    if (key >= get.s.kv || key + (1 << box_log2) <= get.e.first) return r;
    const int col = fast_div(key, p.c.div);
    r.page = get.table[col];
    r.row = key - col * p.c.page;
    r.head = get.h;
    r.any = true;
    return r;
  };
  constexpr uint64_t kAll = KG == 64 ? ~0ull : (1ull << (KG & 63)) - 1;
  // issues the copies; returns the group's keys that may be scored
  auto issue = [&](int st, int stage, const Source& src) -> uint64_t {
    if (st >= steps) {
      if (!TMA) cp_async_commit();
      return 0;
    }
    const uint32_t kd = ring + stage * C::STAGE, vd = kd + KG * C::ROW;
    const int key0 = get.e.lo + get.g * KG, left = get.s.kv - key0;
    uint64_t seen = 0;
    if constexpr (TMA) {
      const bool good_page = src.any && src.page >= 0 && src.page < p.c.pages;
      if (src.any && !good_page) atomicOr(p.err, PAGED_DEVERR_PAGE);
      const uint32_t got = __ballot_sync(0xffffffffu, good_page);
      if (lane == 0) mbar_arrive_expect_tx(bars + stage * 8, (__popc(got) << box_log2) * 128);
      __syncwarp();
      if (good_page)
        tma_box((is_v ? vd : kd) + bx * (KG * 128) + my_row * 128, is_v ? &rp.v : &rp.k, bx * 64,
                src.row, src.head, src.page, bars + stage * 8);
      seen = kAll;
      if (__popc(got) != 2 * per_kv || left < KG) {  // the keys of the boxes that are there
        seen = 0;
        for (int y = 0; y < KG >> box_log2; ++y)
          if (got >> (y * FC) & 1) seen |= ((1ull << ((1 << box_log2) & 63)) - 1) << (y << box_log2);
        if (box_log2 == 6 && (got & 1)) seen = kAll;
        if (left < KG) seen &= left > 0 ? (1ull << left) - 1 : 0;
      }
    } else {
      constexpr int CH = C::ROW / 16;                 // 16-byte pieces of a key
      constexpr int RPI = 32 / CH > 0 ? 32 / CH : 1;  // keys a warp copies at once
#pragma unroll 1
      for (int k0 = 0; k0 < KG; k0 += 16) {
        const int key = key0 + k0 + (lane & 15);
        long long at = -1;
        if (key >= get.e.first && key < get.s.kv) {
          const int col = fast_div(key, p.c.div), page = get.table[col];
          if (page >= 0 && page < p.c.pages)
            at = page * p.c.page_stride + (key - col * p.c.page) * p.c.row_stride +
                 get.h * p.c.head_stride;
          else
            atomicOr(p.err, PAGED_DEVERR_PAGE);
        }
        seen |= (uint64_t)(__ballot_sync(0xffffffffu, at >= 0) & 0xffffu) << k0;
#pragma unroll 4
        for (int i = 0; i < 16 / RPI; ++i) {
          const int r = i * RPI + lane / CH, c = lane % CH;
          const long long o = __shfl_sync(0xffffffffu, at, r);
          const uint32_t nb = o >= 0 ? 16u : 0u;
          const long long e = (o >= 0 ? o : 0) + c * 8;
          cp_async16(kd + C::at(k0 + r, c), p.c.k + e, nb);
          cp_async16(vd + C::at(k0 + r, c), p.c.v + e, nb);
        }
      }
      cp_async_commit();
    }
    return seen;
  };
  constexpr int AHEAD = C::STAGES - 1;
  uint64_t seen[C::STAGES];  // of the next groups: keys that may be scored
  Source src = lookup(0);
#pragma unroll
  for (int st = 0; st < AHEAD; ++st) {
    seen[st] = issue(st, st, src);
    if (st + 1 < steps) advance(get);
    src = lookup(st + 1);
  }

  // In the products' layouts a lane holds keys (and features) g and g + 8 of 16,
  // and rows t2 and t2 + 1 of 8; as an operand's, row g.
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  const int mi = lane >> 3, mr = lane & 7;  // ldmatrix: matrix and row of this lane
  int vis_lo[NB][2], vis_hi[NB][2];         // visible keys of the rows: [lo, hi)
  int strict_lo = 0, strict_hi = 0;         // visible to all rows of the tile
  int r0 = 0, rows = 0;
  float m[NB][2], l[NB][2];
  uint32_t q[NB][D / 16][2];
  float o[NB][D / 16][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 2; ++i) vis_lo[nb][i] = vis_hi[nb][i] = 0;
  bool fresh = true;   // the next group is the first of this warp's part of its item
  bool begun = false;  // ... which began before this warp
  int stage = 0;        // of this group
  uint32_t parity = 0;  // of its barrier
  bool good = true;
#pragma unroll 1
  for (int st = 0; st < steps; ++st) {
    {
      // the copies AHEAD groups on go to the stage read one step ago
      const int nx = stage == 0 ? AHEAD : stage - 1;
      seen[AHEAD] = issue(st + AHEAD, nx, src);
      if (st + AHEAD + 1 < steps) advance(get);
      src = lookup(st + AHEAD + 1);
    }
    if (fresh) {
      fresh = false;
      begun = use.g > 0;
      r0 = use.item / p.c.heads * TILE;
      rows = use.s.nq * p.G;
      const int pos0 = use.s.kv - use.s.nq;
      auto vis = [&](int r, int& a, int& b) {
        const int pos = pos0 + fast_div(min(r0 + r, rows - 1), p.divG);
        b = p.causal || pos < 0 ? min(use.s.kv, pos + 1) : use.s.kv;
        a = p.window > 0 ? window_begin(pos, p.window) : 0;
      };
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        // operand Q^T: row 8 nb + g, features 16 kk + t2, + 1 and + 8, + 9
        const int r = r0 + 8 * nb + g;
        const int tok = r < rows ? fast_div(r, p.divG) : 0;
        const uint16_t* src_q =
            p.q + (r < rows ? (use.s.t0 + tok) * p.q_ts + (use.h * p.G + r - tok * p.G) * p.q_hs : 0);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            q[nb][kk][i] = 0;
            if (r < rows) q[nb][kk][i] = *reinterpret_cast<const uint32_t*>(src_q + kk * 16 + t2 + 8 * i);
          }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          vis(8 * nb + t2 + i, vis_lo[nb][i], vis_hi[nb][i]);
          m[nb][i] = kNegInf;
          l[nb][i] = 0.f;
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nb][d][e] = 0.f;
      }
      int other;  // the first row's last key, the last row's first key
      vis(0, other, strict_hi);
      vis(TILE - 1, strict_lo, other);
    }
    const uint32_t ks = ring + stage * C::STAGE, vs = ks + KG * C::ROW;
    const uint64_t ok = seen[0];
    const int key0 = use.e.lo + use.g * KG;
    const bool edge = ok != kAll || key0 < use.e.first || key0 < strict_lo || key0 + KG > strict_hi;
    if constexpr (TMA) {
      good = copies_wait(bars + stage * 8, parity);
      if (!__all_sync(0xffffffffu, good)) {
        good = false;
        break;
      }
      if (edge) {
        // what lies in rows that no query may see can be NaN, which a weight of
        // zero does not cancel
        const int early = use.e.first - key0;
        uint64_t clear = ~ok & kAll;
        if (early > 0) clear |= early >= KG ? kAll : (1ull << early) - 1;
        if (clear) {
          for (int i = lane; i < KG * (C::ROW / 16); i += 32) {
            const int r = i / (C::ROW / 16), c = i % (C::ROW / 16);
            if (clear >> r & 1)
              *reinterpret_cast<uint4*>(smem + (vs - sm) + C::at(r, c)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();  // before the stage's next copy
        }
      }
    } else {
      cp_async_wait<AHEAD>();
    }
    __syncwarp();
    // ---- S^T: two chains a block where there is only one block
    constexpr int CHAINS = MB * NB >= 4 ? 1 : 2;
    float x[MB][NB][4];
    {
      float sc[CHAINS][MB][NB][4];
#pragma unroll
      for (int ch = 0; ch < CHAINS; ++ch)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[ch][mb][nb][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          // matrices (keys 0-7, k 0-7), (keys 8-15, k 0-7), (0-7, 8-15), (8-15, 8-15)
          uint32_t a[4];
          ldsm4(a, ks + C::at(mb * 16 + (mi & 1) * 8 + mr, 2 * kk + (mi >> 1)));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            mma16816<BF>(sc[kk % CHAINS][mb][nb], a, q[nb][kk][0], q[nb][kk][1]);
        }
      }
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = sc[0][mb][nb][e];
            if (CHAINS == 2) v += sc[CHAINS - 1][mb][nb][e];
            x[mb][nb][e] = v * p.scale_log2;
          }
    }
    if (edge) {
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int kx = mb * 16 + g + 8 * (e >> 1), key = key0 + kx;
            if (!(ok >> kx & 1) || key < vis_lo[nb][e & 1] || key >= vis_hi[nb][e & 1])
              x[mb][nb][e] = kNegInf;
          }
    }
    // ---- running maxima (over the keys: over the lanes of equal t2)
    float now[NB][2];
    bool rise = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = kNegInf;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) v = fmaxf(v, fmaxf(x[mb][nb][i], x[mb][nb][2 + i]));
        now[nb][i] = v;
      }
#pragma unroll
    for (int d = 4; d <= 16; d <<= 1)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          now[nb][i] = fmaxf(now[nb][i], __shfl_xor_sync(0xffffffffu, now[nb][i], d));
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        now[nb][i] = fmaxf(now[nb][i], m[nb][i]);
        rise = rise || now[nb][i] > m[nb][i];
      }
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // (-inf) - (-inf): a row that has seen nothing has nothing to scale
          f[i] = m[nb][i] == now[nb][i] ? 1.f : exp2_approx(m[nb][i] - now[nb][i]);
          l[nb][i] *= f[i];
          m[nb][i] = now[nb][i];
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nb][d][e] *= f[e & 1];
      }
    }
    // ---- P^T as the operand: keys in pairs along a lane, row g
    uint32_t pb[MB][NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const float u0m = m[nb][0] == kNegInf ? 0.f : m[nb][0], u1m = m[nb][1] == kNegInf ? 0.f : m[nb][1];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const float e0 = weight<BF>(x[mb][nb][0] - u0m), e1 = weight<BF>(x[mb][nb][1] - u1m);
        const float e2 = weight<BF>(x[mb][nb][2] - u0m), e3 = weight<BF>(x[mb][nb][3] - u1m);
        l[nb][0] += e0 + e2;
        l[nb][1] += e1 + e3;
        pb[mb][nb][0] = transpose8(pack2<BF>(e0, e1));
        pb[mb][nb][1] = transpose8(pack2<BF>(e2, e3));
      }
    }
    // ---- O^T
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        // matrices (features 0-7, keys 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15)
        uint32_t a[4];
        ldsm4t(a, vs + C::at(mb * 16 + (mi >> 1) * 8 + mr, 2 * d + (mi & 1)));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma16816<BF>(o[nb][d], a, pb[mb][nb][0], pb[mb][nb][1]);
      }
    __syncwarp();  // the stage is read before it is overwritten
    const bool ends = use.g + 1 == use.e.groups;
    if (ends || st + 1 == steps) {
      const bool whole = ends && !begun;
      const long long slot = 2ll * w + (begun ? 0 : 1);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float sum = l[nb][i];
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          constexpr float kDown = BF ? 1.f : 0x1p-15f;  // 2^-kTopWeight
          const int r = 8 * nb + t2 + i;
          if (r0 + r >= rows) continue;
          if (!whole) {
            float* dst = p.part_o + (slot * kRowTile + r) * D + g;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              dst[d * 16] = o[nb][d][i] * kDown;
              dst[d * 16 + 8] = o[nb][d][2 + i] * kDown;
            }
            if (g == 0) p.part_ml[slot * kRowTile + r] = make_float2(m[nb][i], sum * kDown);
          } else {
            const int tok = fast_div(r0 + r, p.divG);
            const int head = use.h * p.G + (r0 + r - tok * p.G);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            uint16_t* dst = p.o + (use.s.t0 + tok) * p.o_ts + head * p.o_hs + g;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              dst[d * 16] = pack1<BF>(o[nb][d][i] * inv);
              dst[d * 16 + 8] = pack1<BF>(o[nb][d][2 + i] * inv);
            }
            if (g == 0 && p.lse)
              p.lse[(long long)(use.s.t0 + tok) * p.Hq + head] =
                  sum == 0.f ? kNegInf : kLn2 * m[nb][i] + logf(sum * kDown);
          }
        }
      fresh = true;
    }
    if (st + 1 < steps) advance(use);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) seen[i] = seen[i + 1];
    if (++stage == C::STAGES) {
      stage = 0;
      parity ^= 1;
    }
  }
  if constexpr (TMA) {
    // (after a wait that gave up: the copies still in flight)
    if (!good) {
      atomicOr(p.err, PAGED_DEVERR_WAIT_TIMEOUT);
      for (int i = 0; i < C::STAGES; ++i) {
        copies_wait(bars + stage * 8, parity);
        if (++stage == C::STAGES) {
          stage = 0;
          parity ^= 1;
        }
      }
    }
  } else {
    cp_async_wait<0>();
  }
}

// Join of a row's parts, in their order: warp w of the row's CTA takes parts
// w, w + W, ...; the warps' sums meet in shared memory.
template <int D, bool BF, int W>
__global__ void __launch_bounds__(32 * W) paged_join_kernel(const AttnParams p) {
  constexpr int E = D / 32;  // features of a lane
  __shared__ float sh_o[W][D];
  __shared__ float sh_l[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long rid = blockIdx.x;
  const int t = (int)(rid / p.Hq), head = (int)(rid - (long long)t * p.Hq);
  // (the batch's arrays were there before the partial results)
  const int n = find_seq(p.b, t);
  const Seq s = load_seq(p.b, max(n, 0));
  // The partial results are there behind this wait.  No CTA leaves before it: this
  // grid must not be over before the first one, whose workspace may be another's
  // from then on.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // new tokens outside every sequence have no partial results
  if (n < 0 || t < s.t0 || t >= s.t0 + s.nq) return;
  // part c of this row: slot (c ? rest + c * step : at), in rows
  long long at, rest, step;
  int parts;
  if (p.chunks > 1) {
    at = rest = rid * p.chunks;
    step = 1;
    parts = p.chunks;
  } else {
    const int r = (t - s.t0) * p.G + head % p.G, tile = r / p.row_tile;
    const Extent e = extent_of(p, s, RowsCfg<D>::KG, p.row_tile);
    const long long U = p.before[p.b.N];
    const long long u = p.before[n] + (long long)(tile * p.c.heads + head / p.G) * e.groups;
    const int warps = (int)min((long long)p.warps, U);
    const int w0 = owner_of(U, warps, u), w1 = owner_of(U, warps, u + e.groups - 1);
    if (w0 == w1) return;  // written by its warp
    at = (2ll * w0 + 1) * kRowTile + r % p.row_tile;
    rest = 2ll * w0 * kRowTile + r % p.row_tile;
    step = 2 * kRowTile;
    parts = w1 - w0 + 1;
  }
  auto slot = [&](int c) { return c == 0 ? at : rest + c * step; };
  float m = kNegInf;
  for (int c = lane; c < parts; c += 32) m = fmaxf(m, p.part_ml[slot(c)].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float u = m == kNegInf ? 0.f : m;
  float l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 8
  for (int c = warp; c < parts; c += W) {
    const float2 x = p.part_ml[slot(c)];
    const float* po = p.part_o + slot(c) * D;
    const float a = exp2_approx(x.x - u);
    l += a * x.y;
    if (x.y != 0.f) {  // (a part without keys need not hold numbers; NaN sums pass)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += a * po[e * 32 + lane];
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sh_o[warp][e * 32 + lane] = acc[e];
  if (lane == 0) sh_l[warp] = l;
  __syncthreads();
  float total = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) total += sh_l[w];
  const float inv = total == 0.f ? 0.f : 1.f / total;
  for (int f = threadIdx.x; f < D; f += 32 * W) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += sh_o[w][f];
    p.o[t * p.o_ts + head * p.o_hs + f] = pack1<BF>(v * inv);
  }
  if (threadIdx.x == 0 && p.lse) p.lse[rid] = total == 0.f ? kNegInf : kLn2 * m + logf(total);
}

template <int D, int NB, bool BF, bool TMA>
cudaError_t rows_launch_t(const RowsParams& rp, cudaStream_t st) {
  using C = RowsCfg<D>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem((const void*)paged_rows_kernel<D, NB, BF, TMA>, C::SMEM, allowed);
  if (e != cudaSuccess) return e;
  return launch_kernel(paged_rows_kernel<D, NB, BF, TMA>, dim3(rp.a.warps / kWarps), dim3(32 * kWarps),
                       C::SMEM, st, rp);
}

template <int D, bool BF>
cudaError_t rows_launch(const AttnParams& p, cudaStream_t st) {
  RowsParams rp;
  rp.a = p;
  int box = RowsCfg<D>::KG;
  while (p.c.page % box) box >>= 1;
  rp.box_log2 = 0;
  while (1 << rp.box_log2 < box) ++rp.box_log2;
  const bool tma = box >= 8 && make_page_map(&rp.k, p.c.k, p.c, 64, box, BF) &&
                   make_page_map(&rp.v, p.c.v, p.c, 64, box, BF);
  if (p.row_tile == 8)
    return tma ? rows_launch_t<D, 1, BF, true>(rp, st) : rows_launch_t<D, 1, BF, false>(rp, st);
  return tma ? rows_launch_t<D, 2, BF, true>(rp, st) : rows_launch_t<D, 2, BF, false>(rp, st);
}

template <int D, bool BF, int W>
cudaError_t join_w(const AttnParams& p, cudaStream_t st) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)((long long)p.b.T * p.Hq));
  c.blockDim = dim3(32 * W);
  c.stream = st;
  // set up while the partial results are still being computed
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, paged_join_kernel<D, BF, W>, p);
}

template <int D, bool BF>
cudaError_t join_launch(const AttnParams& p, cudaStream_t st) {
  // a warp for four parts or so: a row's parts, a kilobyte each at D = 256, are
  // read in as many rounds of latency as a warp has parts
  if (p.parts <= 16) return join_w<D, BF, 4>(p, st);
  return join_w<D, BF, 32>(p, st);
}

}  // namespace

#define PAGED_BY_DIM(FN, ...)                                               \
  switch (p.c.dim) {                                                        \
    case 64: return bf16 ? FN<64, true>(__VA_ARGS__) : FN<64, false>(__VA_ARGS__);    \
    case 128: return bf16 ? FN<128, true>(__VA_ARGS__) : FN<128, false>(__VA_ARGS__); \
    case 256: return bf16 ? FN<256, true>(__VA_ARGS__) : FN<256, false>(__VA_ARGS__); \
  }                                                                         \
  return cudaErrorInvalidValue

cudaError_t launch_paged_rows(const AttnParams& p, bool bf16, cudaStream_t st) {
  PAGED_BY_DIM(rows_launch, p, st);
}
cudaError_t launch_paged_join(const AttnParams& p, bool bf16, cudaStream_t st) {
  PAGED_BY_DIM(join_launch, p, st);
}

}  // namespace moe
