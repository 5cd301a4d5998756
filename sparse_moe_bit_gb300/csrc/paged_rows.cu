// Attention of a few query rows of a key/value head over the paged cache, and
// the join of results that were split over the keys (include/paged.h).
//
// The G query heads that share a key/value head and the sequence's new tokens
// form the rows of one small matrix: row r is token r / G, head r % G of the
// group.  An item is 16 rows (one mma tile) of a sequence over all of their
// keys, so that every key and value is read from HBM once for the whole group.
//   S = Q K^T, m' = max(m, rowmax S), P = 2^(S - m'), l = l 2^(m - m') + sum P,
//   O = O 2^(m - m') + P V                         (S in log2 units, all fp32)
//
// Bound: HBM (2 bytes x 2 D per key against 2 x 4 D x rows operations).  What
// counts is bytes in flight and an even share for every SM, so the work is cut
// into groups of 16 keys, the groups of all items stand in one row, and each of
// the launch's warps takes the same number of them in sequence, across items:
// no warp ever waits for another.  It streams its groups through a ring of its
// own, filled by 16-byte asynchronous copies two or more groups ahead (page
// numbers one further), and keeps m, l and O of its 16 rows in registers.  An
// item that one warp covers is written at once; of the others every warp leaves
// O, m and l in a slot -- a warp has at most two such items, its first and its
// last -- and a second kernel joins them in order, which makes the result
// independent of timing.  (Chunks of keys fixed on the host, a CTA each, gave
// 72 % of the copy bandwidth on 64 ragged contexts up to 8192: the last wave
// ran half empty.)  The product of 16 rows by mma.sync (m16n8k16) needs a tenth
// of the rate at which keys arrive; wider row tiles go to the tcgen05 kernel.
// Rows of a page that lie behind the sequence's end, or whose page number is
// bad, are never read: the copy fills them with zeros and the score is masked.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kWarps = kRowWarps;  // of a CTA
constexpr int kGroup = 16;  // keys of a warp's step

template <int D>
struct RowsCfg {
  static constexpr int ROW = 2 * D;  // bytes of a key
  static constexpr int STAGES = D == 64 ? 4 : 3;
  static constexpr int STAGE = 2 * kGroup * ROW;  // keys and values of a group
  static constexpr int RING = kWarps * STAGES * STAGE;
  static constexpr int OFF_Q = RING;
  static constexpr int OFF_BAR = OFF_Q + kWarps * kRowTile * ROW;  // per warp and stage
  static constexpr int SMEM = OFF_BAR + kWarps * STAGES * 8 + 1024;
  static_assert(SMEM + 1100 <= 232448, "shared memory budget");  // (the rest: static)
};
// 16 rows of D features in shared memory: blocks of 64 features, rows of 128
// bytes, the 16-byte pieces of a row swizzled by the row -- the 128-byte swizzle
// of TMA, and free of bank conflicts for ldmatrix.  Offset of piece c of row r:
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  return (c >> 3) * (kGroup * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Tensor maps over the cache's keys and values (innermost first): feature, row
// of a page, head, page; boxes of 64 features x `box` (16 or 8) rows.
struct RowsParams {
  AttnParams a;
  CUtensorMap k, v;
  int box;
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

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.69314718055994530942f;

// The items of one sequence: `items` (row tile, key/value head) pairs of
// `groups` groups each, over the keys [lo, kv).  A sequence with rows has at
// least one group an item, so that rows without keys are written too.
struct Extent {
  int lo, first, groups, items;  // first: the first key that a row may see
};
__device__ __forceinline__ Extent extent_of(const AttnParams& p, const Seq& s) {
  Extent e;
  const int rows = s.nq * p.G;
  e.first = p.window > 0 ? max(0, s.kv - s.nq - p.window + 1) : 0;
  e.lo = e.first & ~(kGroup - 1);  // groups do not straddle pages that hold whole ones
  e.groups = max((s.kv - e.lo + kGroup - 1) / kGroup, 1);
  e.items = (rows + kRowTile - 1) / kRowTile * p.c.heads;
  return e;
}
// warp w of W takes the groups [share(w), share(w + 1)) of U
__device__ __forceinline__ long long share_of(long long U, int W, int w) { return U * w / W; }
// ... and group u is warp owner(u)'s
__device__ __forceinline__ int owner_of(long long U, int W, long long u) {
  return (int)(((u + 1) * W - 1) / U);
}

// TMA: a group is copied as boxes of the pages' rows, a lane each; otherwise
// (pages that no box of 8 rows divides) by 16-byte copies.
template <int D, bool BF, bool TMA>
__global__ void __launch_bounds__(32 * kWarps)
    paged_rows_kernel(const __grid_constant__ RowsParams rp) {
  const AttnParams& p = rp.a;
  using C = RowsCfg<D>;
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
    const Extent e = extent_of(p, load_seq(p.b, n));
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
      const Extent e = extent_of(p, load_seq(p.b, n));
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
      c.e = extent_of(p, c.s);
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
  const uint32_t qs = sm + C::OFF_Q + warp * kRowTile * C::ROW;
  const uint32_t ring = sm + warp * C::STAGES * C::STAGE;
  const uint32_t bars = sm + C::OFF_BAR + warp * C::STAGES * 8;
  if (TMA) {
    if (lane < C::STAGES) mbar_init(bars + lane * 8, 1);
    fence_mbar_init();
    __syncwarp();
  }

  // ---- the ring.  TMA: lane l copies box l of a group (blocks of 64 features
  // side by side, keys then values; at most 16 boxes).  Else: lane l (and l + 16)
  // addresses key l.  Where a lane's copy of group `st` comes from:
  constexpr int FC = D / 64;
  const int box = TMA ? rp.box : 1, per_kv = FC * (kGroup / box);  // boxes of the keys
  const bool is_v = TMA && lane >= per_kv;
  const int bx = (lane - (is_v ? per_kv : 0)) % FC, by = (lane - (is_v ? per_kv : 0)) / FC;
  const bool copies = TMA ? lane < 2 * per_kv : true;
  const int my_row = TMA ? by * box : (lane & 15);
  struct Source {
    int page, row, head;
    bool any;  // something to copy
  };
  // (the page number is not looked at before the copies are issued, a step later:
  // its load is then never waited for)
  auto lookup = [&](int st) -> Source {
    Source r{-1, 0, 0, false};
    const int key = get.e.lo + get.g * kGroup + my_row;
    if (!copies || st >= steps || key >= get.s.kv || key + box <= get.e.first) return r;
    const int col = fast_div(key, p.c.div);
    r.page = get.table[col];
    r.row = key - col * p.c.page;
    r.head = get.h;
    r.any = true;
    return r;
  };
  // issues the copies; returns the group's keys that may be scored
  auto issue = [&](int st, int stage, const Source& src) -> uint32_t {
    if (st >= steps) {
      if (!TMA) cp_async_commit();
      return 0;
    }
    const bool good_page = src.any && src.page >= 0 && src.page < p.c.pages;
    if (src.any && !good_page) atomicOr(p.err, PAGED_DEVERR_PAGE);
    const uint32_t kd = ring + stage * C::STAGE, vd = kd + kGroup * C::ROW;
    if constexpr (TMA) {
      const uint32_t got = __ballot_sync(0xffffffffu, good_page);
      if (lane == 0) mbar_arrive_expect_tx(bars + stage * 8, __popc(got) * box * 128);
      __syncwarp();
      if (good_page)
        tma_box((is_v ? vd : kd) + bx * (kGroup * 128) + my_row * 128, is_v ? &rp.v : &rp.k, bx * 64,
                src.row, src.head, src.page, bars + stage * 8);
      // keys of the boxes that hold some, up to the sequence's end
      uint32_t seen = box == 16 ? (got & 1 ? 0xffffu : 0)
                                : ((got & 1 ? 0x00ffu : 0) | (got >> FC & 1 ? 0xff00u : 0));
      const int left = get.s.kv - (get.e.lo + get.g * kGroup);
      if (left < kGroup) seen &= left > 0 ? (1u << left) - 1 : 0;
      return seen;
    } else {
      const long long at = !good_page ? -1
                                        : src.page * p.c.page_stride + src.row * p.c.row_stride +
                                              src.head * p.c.head_stride;
      constexpr int CH = C::ROW / 16;                 // 16-byte pieces of a key
      constexpr int RPI = 32 / CH > 0 ? 32 / CH : 1;  // keys a warp copies at once
#pragma unroll 4
      for (int i = 0; i < kGroup / RPI; ++i) {
        const int r = i * RPI + lane / CH, c = lane % CH;
        const long long o = __shfl_sync(0xffffffffu, at, r);
        const uint32_t nb = o >= 0 ? 16u : 0u;
        const long long e = (o >= 0 ? o : 0) + c * 8;
        cp_async16(kd + piece_at(r, c), p.c.k + e, nb);
        cp_async16(vd + piece_at(r, c), p.c.v + e, nb);
      }
      cp_async_commit();
      return __ballot_sync(0xffffffffu, at >= 0) & 0xffffu;
    }
  };
  constexpr int AHEAD = C::STAGES - 1;
  uint32_t seen[C::STAGES];  // of the next groups: keys that may be scored
  Source src = lookup(0);
#pragma unroll
  for (int st = 0; st < AHEAD; ++st) {
    seen[st] = issue(st, st, src);
    if (st + 1 < steps) advance(get);
    src = lookup(st + 1);
  }

  // per-thread rows: g and g + 8 of the tile
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  const int mi = lane >> 3, mr = lane & 7;  // ldmatrix: matrix and row of this lane
  int hiA = 0, hiB = 0, loA = 0, loB = 0;   // visible keys of the two rows: [lo, hi)
  int strict_lo = 0, strict_hi = 0;         // visible to all rows of the tile
  int r0 = 0, rows = 0, h = 0;
  float mA = kNegInf, mB = kNegInf, lA = 0.f, lB = 0.f;
  float o[D / 8][4];
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
      h = use.h;
      r0 = use.item / p.c.heads * kRowTile;
      rows = use.s.nq * p.G;
      // Q rows into shared memory, 16-byte chunks swizzled by the row
      constexpr int CH = C::ROW / 16;
#pragma unroll 4
      for (int i = lane; i < kRowTile * CH; i += 32) {
        const int r = i / CH, c = i % CH;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r0 + r < rows) {
          const int tok = fast_div(r0 + r, p.divG);
          v = *reinterpret_cast<const uint4*>(p.q + (use.s.t0 + tok) * p.q_ts +
                                              (h * p.G + r0 + r - tok * p.G) * p.q_hs + c * 8);
        }
        *reinterpret_cast<uint4*>(smem + C::OFF_Q + warp * kRowTile * C::ROW + piece_at(r, c)) = v;
      }
      auto range = [&](int r, int& a, int& b) {
        const int pos = use.s.kv - use.s.nq + fast_div(min(r0 + r, rows - 1), p.divG);
        b = p.causal ? min(use.s.kv, pos + 1) : use.s.kv;
        a = p.window > 0 ? pos - p.window + 1 : 0;
      };
      range(g, loA, hiA);
      range(g + 8, loB, hiB);
      int last;  // the first row's last key, the last row's first key
      range(0, last, strict_hi);
      range(kRowTile - 1, strict_lo, last);
      mA = mB = kNegInf;
      lA = lB = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    }
    const uint32_t ks = ring + stage * C::STAGE, vs = ks + kGroup * C::ROW;
    const uint32_t ok = seen[0];
    if constexpr (TMA) {
      good = copies_wait(bars + stage * 8, parity);
      if (!__all_sync(0xffffffffu, good)) {
        good = false;
        break;
      }
      // Rows behind the sequence's end (or before its window, or of a bad page)
      // can hold anything, NaN included, which a weight of zero does not cancel:
      // values of keys that no row may see are zeroed.
      const int early = max(use.e.first - (use.e.lo + use.g * kGroup), 0);
      uint32_t clear = ~ok & 0xffffu;
      if (early > 0) clear |= (1u << min(early, 16)) - 1;
      if (clear) {
        for (int i = lane; i < kGroup * (C::ROW / 16); i += 32) {
          const int r = i / (C::ROW / 16), c = i % (C::ROW / 16);
          if (clear >> r & 1)
            *reinterpret_cast<uint4*>(smem + (vs - sm) + piece_at(r, c)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // before the stage's next copy
      }
    } else {
      cp_async_wait<AHEAD>();
    }
    __syncwarp();
    // S: two blocks of 8 keys, four accumulators each to shorten the chains
    float sc[2][4][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[i][j][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t a[4], b[4];
      // A: matrices (rows 0-7, k 0-7), (rows 8-15, k 0-7), (0-7, 8-15), (8-15, 8-15)
      {
        const int r = (mi & 1) * 8 + mr, c = 2 * kk + (mi >> 1);
        ldsm4(a, qs + piece_at(r, c));
      }
      {
        const int r = (mi >> 1) * 8 + mr, c = 2 * kk + (mi & 1);
        ldsm4(b, ks + piece_at(r, c));
      }
      mma16816<BF>(sc[0][kk & 3], a, b[0], b[1]);
      mma16816<BF>(sc[1][kk & 3], a, b[2], b[3]);
    }
    const int key0 = use.e.lo + use.g * kGroup;
    float x[2][4];
#pragma unroll
    for (int nb = 0; nb < 2; ++nb)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[nb][e] = ((sc[nb][0][e] + sc[nb][1][e]) + (sc[nb][2][e] + sc[nb][3][e])) * p.scale_log2;
    if (ok != 0xffffu || key0 < strict_lo || key0 + kGroup > strict_hi) {
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int kx = nb * 8 + t2 + (e & 1), key = key0 + kx;
          const bool vis = (ok >> kx & 1) && (e < 2 ? (key >= loA && key < hiA)
                                                    : (key >= loB && key < hiB));
          if (!vis) x[nb][e] = kNegInf;
        }
      }
    }
    float nA = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
    float nB = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
      nA = fmaxf(nA, __shfl_xor_sync(0xffffffffu, nA, d));
      nB = fmaxf(nB, __shfl_xor_sync(0xffffffffu, nB, d));
    }
    nA = fmaxf(mA, nA);
    nB = fmaxf(mB, nB);
    if (__any_sync(0xffffffffu, nA > mA || nB > mB)) {
      // (-inf) - (-inf): a row that has seen nothing has nothing to scale
      const float fA = mA == nA ? 1.f : exp2_approx(mA - nA);
      const float fB = mB == nB ? 1.f : exp2_approx(mB - nB);
      lA *= fA;
      lB *= fB;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= fA;
        o[i][1] *= fA;
        o[i][2] *= fB;
        o[i][3] *= fB;
      }
      mA = nA;
      mB = nB;
    }
    const float uA = mA == kNegInf ? 0.f : mA, uB = mB == kNegInf ? 0.f : mB;
    uint32_t pa[4];
    {
      float e0[4], e1[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        e0[e] = exp2_approx(x[0][e] - (e < 2 ? uA : uB));
        e1[e] = exp2_approx(x[1][e] - (e < 2 ? uA : uB));
      }
      lA += (e0[0] + e0[1]) + (e1[0] + e1[1]);
      lB += (e0[2] + e0[3]) + (e1[2] + e1[3]);
      pa[0] = pack2<BF>(e0[0], e0[1]);
      pa[1] = pack2<BF>(e0[2], e0[3]);
      pa[2] = pack2<BF>(e1[0], e1[1]);
      pa[3] = pack2<BF>(e1[2], e1[3]);
    }
#pragma unroll
    for (int nn = 0; nn < D / 16; ++nn) {
      uint32_t b[4];
      const int r = (mi & 1) * 8 + mr, c = 2 * nn + (mi >> 1);
      ldsm4t(b, vs + piece_at(r, c));
      mma16816<BF>(o[2 * nn], pa, b[0], b[1]);
      mma16816<BF>(o[2 * nn + 1], pa, b[2], b[3]);
    }
    __syncwarp();  // the stage and Q are read before they are overwritten
    const bool ends = use.g + 1 == use.e.groups;
    if (ends || st + 1 == steps) {
#pragma unroll
      for (int d = 1; d <= 2; d <<= 1) {
        lA += __shfl_xor_sync(0xffffffffu, lA, d);
        lB += __shfl_xor_sync(0xffffffffu, lB, d);
      }
      const bool whole = ends && !begun;
      const long long slot = 2ll * w + (begun ? 0 : 1);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = g + 8 * half;
        const float m = half ? mB : mA, l = half ? lB : lA;
        if (r0 + r >= rows) continue;
        if (!whole) {
          float* d = p.part_o + (slot * kRowTile + r) * D + t2;
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2*>(d + i * 8) = make_float2(o[i][2 * half], o[i][2 * half + 1]);
          if ((lane & 3) == 0) p.part_ml[slot * kRowTile + r] = make_float2(m, l);
        } else {
          const int tok = fast_div(r0 + r, p.divG);
          const int head = h * p.G + (r0 + r - tok * p.G);
          const float inv = l == 0.f ? 0.f : 1.f / l;
          uint16_t* d = p.o + (use.s.t0 + tok) * p.o_ts + head * p.o_hs + t2;
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<uint32_t*>(d + i * 8) =
                pack2<BF>(o[i][2 * half] * inv, o[i][2 * half + 1] * inv);
          if ((lane & 3) == 0 && p.lse)
            p.lse[(long long)(use.s.t0 + tok) * p.Hq + head] =
                l == 0.f ? kNegInf : kLn2 * m + logf(l);
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
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long rid = blockIdx.x;
  const int t = (int)(rid / p.Hq), head = (int)(rid - (long long)t * p.Hq);
  // new tokens outside every sequence have no partial results
  const int n = find_seq(p.b, t);
  if (n < 0) return;
  const Seq s = load_seq(p.b, n);
  if (t < s.t0 || t >= s.t0 + s.nq) return;
  // part c of this row: slot (c ? rest + c * step : at), in rows
  long long at, rest, step;
  int parts;
  if (p.chunks > 1) {
    at = rest = rid * p.chunks;
    step = 1;
    parts = p.chunks;
  } else {
    const int r = (t - s.t0) * p.G + head % p.G, tile = r / kRowTile;
    const Extent e = extent_of(p, s);
    const long long U = p.before[p.b.N];
    const long long u = p.before[n] + (long long)(tile * p.c.heads + head / p.G) * e.groups;
    const int warps = (int)min((long long)p.warps, U);
    const int w0 = owner_of(U, warps, u), w1 = owner_of(U, warps, u + e.groups - 1);
    if (w0 == w1) return;  // written by its warp
    at = (2ll * w0 + 1) * kRowTile + r % kRowTile;
    rest = 2ll * w0 * kRowTile + r % kRowTile;
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
#pragma unroll 4
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

template <int D, bool BF, bool TMA>
cudaError_t rows_launch_t(const RowsParams& rp, cudaStream_t st) {
  using C = RowsCfg<D>;
  static bool attr_set = false;
  if (!attr_set) {
    const cudaError_t e = cudaFuncSetAttribute(
        paged_rows_kernel<D, BF, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_set = true;
  }
  return launch_kernel(paged_rows_kernel<D, BF, TMA>, dim3(rp.a.warps / kWarps), dim3(32 * kWarps),
                       C::SMEM, st, rp);
}

template <int D, bool BF>
cudaError_t rows_launch(const AttnParams& p, cudaStream_t st) {
  RowsParams rp;
  rp.a = p;
  rp.box = p.c.page % 16 == 0 ? 16 : 8;
  if (p.c.page % 8 == 0 && make_page_map(&rp.k, p.c.k, p.c, 64, rp.box, BF) &&
      make_page_map(&rp.v, p.c.v, p.c, 64, rp.box, BF))
    return rows_launch_t<D, BF, true>(rp, st);
  return rows_launch_t<D, BF, false>(rp, st);
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
  return join_w<D, BF, 4>(p, st);
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
