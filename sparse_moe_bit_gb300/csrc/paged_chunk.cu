// Attention of many query rows over the paged cache on the tensor cores
// (include/paged.h): chunks of new tokens, from a few tokens of a wide head
// group to whole prompts.
//
// A pair of CTAs (a cluster of two, tcgen05 cta_group::2) takes 256 rows -- row
// r is token r / G, head r % G of the G query heads on one key/value head --
// and walks its visible keys in tiles of 128, with the running softmax of
//   S = Q K^T, m' = max(m, rowmax S), P = 2^(S - m'), l = l 2^(m - m') + sum P,
//   O = O 2^(m - m') + P V        (S in log2 units; S, m, l, O fp32)
// Each CTA holds 128 of the rows: its Q in shared memory, its O (D columns) and
// S buffers (128 columns each) in TMEM: two at D = 256, which fill the 512
// columns, three below.
// The pair shares the operands: of a tile each CTA loads 64 keys (half of B's
// columns in Q K^T) and half of every value's features (half of B's columns in
// P V), so that a byte of the cache enters one SM for 256 rows.  P goes back to
// TMEM over the S it came from (16-bit, the MMA's A operand); V is read from
// shared memory as it lies in the cache, [key][feature] (the "MN-major" form).
//
// Bound: the tensor cores (4 D operations per row and key).  Their two products
// of tile j and the softmax of tile j + 1 overlap: the order of issue is
// QK(0), QK(1), PV(0), QK(2), PV(1), ... (one more ahead with three S buffers).
// Two groups of eight warps take the even and the odd tiles, a thread half a row,
// so that one group's exponentials run while the other waits or reduces; they pass
// the reference maximum on from tile to tile.  It only moves when it rises by more
// than 2^8 (weights then stay below 2^8, which fp32 sums and 16-bit weights carry
// without loss), so that O in TMEM is hardly ever rescaled.  (fp16: P = 2^(S - m' + 7),
// so that small weights stay in the type's range, off by half a step or 2^-32 of the
// reference's; l and O likewise, with m' - 7 as their reference.)
//
// Measured, bf16, 16 query and 2 key/value heads: D = 256, 4096 new tokens over 32768
// keys 1.14 ms at 2070 MHz, 1.80 PFLOP/s (0.95 of cuBLAS's burst; 1.21 ms at the 1.82
// GHz that the power limit leaves launches back to back), 2048 over 16384 1.79 PFLOP/s,
// tensor pipe 88 % active; 2048 over 16384 with D = 128 1.44 PFLOP/s and with D = 64
// 0.75, in the same time a tile.  There no unit is full (D = 128: tensor 67 %, issue
// 56 %, ALU 40 %, XU 35 %; D = 64: tensor 34 %, the others alike): a tile's chain of
// scores out of TMEM, maxima, exponentials, weights back and hand-over bounds it, which
// the two groups overlap in part.  Tried for the small heads and slower: P in TMEM
// columns of its own with a second warp that issues P V (D = 128 1.32, D = 64 0.66: the
// two warps' MMAs interleave and each product finishes late), and with a whole row a
// thread at 200 registers (1.37 and 0.71).
//
// Warps: 0 copies keys, 2 copies values, 1 issues the MMAs (the even CTA's),
// 4..19 softmax, correction and epilogue.  Every wait is bounded.  The copies
// are TMA boxes of up to 64 rows of a page x 64 features, a lane each, into the
// operands' swizzled layouts (copying the same by 16-byte cp.async took one
// warp 4500 cycles a tile at D = 256 where the products take 2048).  A box that
// also holds keys outside the chunk's is loaded whole for K (those scores are
// masked) but row by row for V: what lies there may be NaN, which a weight of
// zero does not cancel.  A bad page number becomes the number behind the last
// page, where TMA fills in zeros, and its scores are masked.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 640;
constexpr int kSoftWarp0 = 4, kSoftWarps = 16;  // two groups of two halves of a row
constexpr int kTileKeys = 128;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRise = 8.f;  // log2 units the maximum may lag behind
// fp16's weights are up to 2^(kShift + kRise), the type's range.  (A shift of 12 with a
// rise of 3 kept five bits more of small weights but rescaled O at every other tile:
// 2048 tokens over 16K keys, 256 features, 300 -> 513 us.)
template <bool BF>
constexpr float kShift = BF ? 0.f : kTopWeight<BF> - kRise;

// log2 units of a reference whose fp32 step is small enough for x c - mc with mc rounded;
// past it scores are taken relative to the reference first
constexpr float kFar = 4096.f;

template <int D>
struct ChunkCfg {
  static constexpr int Q_BYTES = 128 * D * 2;
  static constexpr int STAGE = 128 * D;  // 64 keys, or half the features of 128 values
  // S buffers in TMEM beside O's D columns, and stages of K and of V: everything
  // of a tile moves on together (see Bars)
  static constexpr int NS = D == 256 ? 2 : 3;
  static constexpr int OFF_K = Q_BYTES;
  static constexpr int OFF_V = OFF_K + NS * STAGE;
  static constexpr int OFF_BAR = OFF_V + NS * STAGE;
  static constexpr int NUM_BARS = 2 + 3 * NS;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NUM_BARS;
  static constexpr int OFF_REF = (OFF_MISC + 64 + 15) / 16 * 16;  // float [4][128]
  static constexpr int OFF_MAX = OFF_REF + 4 * 128 * 4;           // float [4][2][128]
  static constexpr int OFF_ML = 0;  // float4 [4][128], over Q, which is done with then
  static constexpr int USED = OFF_MAX + 8 * 128 * 4 + 1024;
  // never two CTAs on an SM: each takes all of TMEM, and two pairs that held one
  // SM each would wait for one another
  static constexpr int SMEM = USED > 120000 ? USED : 120000;
  static_assert(SMEM <= 232448, "shared memory budget");
  static constexpr int S_COL = 512 - 128 * NS;  // TMEM: O at 0, S buffers at the end
  static_assert(D <= S_COL, "TMEM budget");
};

// Barriers (the even CTA's unless said otherwise; t % NS in brackets).  The
// issuing warp waits once and commits once a tile -- every wait, test or commit
// costs it some 150 cycles, and the tensor core runs dry meanwhile:
//   ready(j)  P(j) of both CTAs is in TMEM, V(j) and K(j + NS) in shared memory
//   moved(t)  (both CTAs) QK(t) has completed, and with it P V(t - NS), issued
//             before it: S(t) can be read; the stages of K(t) and V(t - NS) are
//             free; O holds the products up to tile t - NS
//   k_first   K(t), t < NS
template <int D>
struct Bars {
  using C = ChunkCfg<D>;
  uint32_t base;
  __device__ uint32_t q_full() const { return base; }
  __device__ uint32_t drain() const { return base + 8; }
  __device__ uint32_t moved(int s) const { return base + 8 * (2 + s); }
  __device__ uint32_t ready(int s) const { return base + 8 * (2 + C::NS + s); }
  __device__ uint32_t k_first(int s) const { return base + 8 * (2 + 2 * C::NS + s); }
};

// (CLUSTER: acquires what another CTA's threads wrote to shared memory by plain
// or asynchronous copies; what TMA wrote or lies in TMEM needs no more than the
// default, which costs the MMA warp some hundred cycles less a wait)
template <bool CLUSTER>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  if constexpr (!CLUSTER) return mbar_try_wait_sleep(bar, parity);
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}
// Arrive on an mbarrier of any CTA of the cluster, releasing this thread's
// writes to the cluster.
__device__ __forceinline__ void arrive_release_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// Waits for the copies counted on `bar`, whatever else has given up.
__device__ __forceinline__ void copies_done(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_sleep(bar, parity))
    if (globaltimer_ns() - t0 > kWaitLimitNs) return;
}

// The whole warp waits; false when the limit has passed or another wait of the
// CTA has given up.
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          int* err) {
  bool ok = try_wait<CLUSTER>(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    ok = ok || try_wait<CLUSTER>(bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    int bail = 0;
    if ((threadIdx.x & 31) == 0) bail = (*abort_flag || globaltimer_ns() - t0 > kWaitLimitNs);
    if (__shfl_sync(0xffffffffu, bail, 0)) {
      if ((threadIdx.x & 31) == 0) {
        *abort_flag = 1;
        atomicOr(err, PAGED_DEVERR_WAIT_TIMEOUT);
      }
      return false;
    }
  }
}

// Four MMAs (K = 64) of D (+)= A[smem] * B[smem]^T over the pair, M = 256, both
// operands advancing by 32 bytes.  Warp-wide: every lane makes the call, one
// elected lane issues; one block for all four, so that the election and the
// moves of the operands to uniform registers are paid once.
__device__ __forceinline__ void mma_ss_x4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\tsetp.eq.b32 p, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Four MMAs (K = 64) of D (+)= A[tmem] * B[smem], A advancing by 8 columns and
// B's descriptor by STEP.
template <int STEP>
__device__ __forceinline__ void mma_ts_x4(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.s32 a, %1, 8;\n\tadd.s64 b, %2, %5;\n\tsetp.eq.b32 p, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %3, p;\n\t"
      "add.s32 a, %1, 16;\n\tadd.s64 b, %2, %6;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %3, p;\n\t"
      "add.s32 a, %1, 24;\n\tadd.s64 b, %2, %7;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "n"(STEP), "n"(2 * STEP), "n"(3 * STEP)
      : "memory");
}

// Descriptor of a B tile stored [K][N] with N contiguous: rows (one K each) of
// `row` bytes, 128 (swizzle over 8 rows of 128 bytes) or 64 (over 8 rows of 64
// bytes).  Stride offset: 8 rows; leading offset: from one row's width of N to
// the next.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t addr, int row, int lead) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(row * 8 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)(row == 128 ? 2 : 4) << 61);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
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
// x rounded to the 16-bit type
template <bool BF>
__device__ __forceinline__ float round16(float x) {
  if constexpr (BF) return __bfloat162float(__float2bfloat16_rn(x));
  else return __half2float(__float2half_rn(x));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// pairs of fp32 in one 64-bit register
__device__ __forceinline__ uint64_t pack_u2(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack_f2(float a, float b) {
  return pack_u2(__float_as_uint(a), __float_as_uint(b));
}
__device__ __forceinline__ void unpack_f2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void pair_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Barriers of a lane quarter: the one of group g's tile counts its two halves'
// warps, which wait, and the warp of the other group that hands on the reference.
__device__ __forceinline__ void tile_arrive(int g, int q) {
  asm volatile("bar.arrive %0, 96;" ::"r"(5 + g * 4 + q) : "memory");
}
__device__ __forceinline__ void tile_wait(int g, int q) {
  asm volatile("bar.sync %0, 96;" ::"r"(5 + g * 4 + q) : "memory");
}
// whether any thread of the softmax warps says so
__device__ __forceinline__ bool softmax_any(int v) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 13, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(v), "n"(32 * kSoftWarps)
      : "memory");
  return r != 0;
}
// the four warps that share a lane quarter's rows
__device__ __forceinline__ void quarter_sync(int q) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory");
}

// Tensor maps over the cache's keys and values (innermost first): feature, row
// of a page, head, page; boxes of `box` rows x 64 features (keys) or x 64 (32 at
// D = 64) features (values), in the operands' swizzles.
struct ChunkParams {
  AttnParams a;
  CUtensorMap k, v;
  int box_log2;  // rows of a box: a power of two that divides the page and 64, >= 8
};

__device__ __forceinline__ void tma_box_pair(uint32_t dst, const CUtensorMap* tm, int f, int r,
                                             int h, int pg, uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(tm), "r"(f), "r"(r), "r"(h), "r"(pg), "r"(bar_cluster)
      : "memory");
}

// TMA: whole boxes of the cache are copied by the tensor memory accelerator;
// otherwise (pages that no box of 8 rows divides) by 16-byte copies alone.
template <int D, bool BF, bool TMA>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ ChunkParams cp) {
  const AttnParams& p = cp.a;
  using C = ChunkCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ int sh_find[4], sh_scan[kThreads / 32];
  const uint32_t sm = smem_u32(smem);
  const Bars<D> B{sm + C::OFF_BAR};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  // barriers and TMEM, while the other warps look for the tile
  if (warp == 2 && lane == 0) {
    mbar_init(B.q_full(), 2 * kSoftWarps);
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(B.moved(i), 1);
      // one softmax group's warps of both CTAs, and each CTA's copying warps
      mbar_init(B.ready(i), kSoftWarps + 4);
      mbar_init(B.k_first(i), 2);
    }
    mbar_init(B.drain(), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  auto leave = [&]() {  // every warp of both CTAs
    tc_fence_before();
    __syncthreads();
    pair_sync_all();  // no CTA leaves while the other may still arrive on its barriers
    if (warp == 1) {
      tc_fence_after();
      tmem_dealloc_pair(*tmem_slot, 512);
    }
  };

  int bid = blockIdx.x >> 1;
  const int ck = bid % p.chunks;
  bid /= p.chunks;
  const int h = bid % p.c.heads;
  const int want = bid / p.c.heads;  // the want-th row tile of the batch

  // ---- which sequence's which tile: running sum of the sequences' tile counts
  if (threadIdx.x == 0) sh_find[0] = -1;
  int before = 0;
  for (int n0 = 0; n0 < p.b.N; n0 += kThreads) {
    const int n = n0 + threadIdx.x;
    const int nt = n < p.b.N ? (load_seq(p.b, n).nq * p.G + 255) / 256 : 0;
    int inc = nt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += o;
    }
    __syncthreads();  // sh_scan of the step before is read
    if (lane == 31) sh_scan[warp] = inc;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) inc += sh_scan[w];
      total += sh_scan[w];
    }
    inc += before;
    if (want < inc && want >= inc - nt) {
      sh_find[0] = n;
      sh_find[1] = nt - 1 - (want - (inc - nt));  // last tile first: it sees the most keys
    }
    before += total;
    if (want < before) break;  // uniform
  }
  tc_fence_before();
  __syncthreads();
  const int n = sh_find[0];
  if (n < 0) {  // uniform over the pair: both CTAs look for the same tile
    leave();
    return;
  }
  const int tile = sh_find[1];
  const Seq s = load_seq(p.b, n);
  const int rows = s.nq * p.G;
  const int r0 = tile * 256, r1 = min(r0 + 256, rows);
  const int2 kr = key_range(p, s, r0, r1);
  const int span = kr.y - kr.x;
  const long long c0 = (long long)ck * p.chunk;
  // keys of this chunk [lo, hi), in tiles from `first` (a box's boundary) on
  const int lo = kr.x + (int)min(c0, (long long)span);
  const int hi = ck == p.chunks - 1 ? kr.y : kr.x + (int)min(c0 + p.chunk, (long long)span);
  const int first = TMA ? lo & ~63 : lo;
  const int nb = hi > lo ? (hi - first + kTileKeys - 1) / kTileKeys : 0;
  const int32_t* table = p.b.table + n * p.b.table_stride;

  // this thread's row in the softmax warps (the other warps: unused)
  const int quarter = warp & 3, half = ((warp - kSoftWarp0) >> 2) & 1;
  const int group = (warp - kSoftWarp0) >> 3;
  const int trow = quarter * 32 + lane;
  const int row = r0 + rank * 128 + trow;
  const bool valid = row < r1;
  const int tok = valid ? fast_div(row, p.divG) : 0;
  const int head = h * p.G + (valid ? row - tok * p.G : 0);
  const long long rid = (long long)(s.t0 + tok) * p.Hq + head;

  if (nb == 0) {  // nothing to see in this chunk (uniform over the pair)
    if (warp >= kSoftWarp0 && valid) {
      const int part = half + 2 * group;  // a quarter of the features
      if (p.chunks > 1) {
        if (part == 0) p.part_ml[rid * p.chunks + ck] = make_float2(kNegInf, 0.f);
      } else {
        uint16_t* o = p.o + (s.t0 + tok) * p.o_ts + head * p.o_hs + part * (D / 4);
        for (int f = 0; f < D / 4; f += 8) *reinterpret_cast<uint4*>(o + f) = make_uint4(0, 0, 0, 0);
        if (part == 0 && p.lse) p.lse[rid] = kNegInf;
      }
    }
    leave();
    return;
  }

  pair_sync_all();  // the other CTA's barriers are there before anything arrives on them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // element offset of key `key`'s row in the cache, -1: none
  auto lookup = [&](int key) -> long long {
    if (key >= hi) return -1;
    const int col = fast_div(key, p.c.div);
    const int pg = table[col];
    if (pg < 0 || pg >= p.c.pages) return -1;
    return pg * p.c.page_stride + (key - col * p.c.page) * p.c.row_stride;
  };

  // Registers: 96 x 640 at launch = 64 x 128 + 104 x 512 (a thread of the softmax
  // holds half of a row's scores of a tile).
  if (warp < kSoftWarp0) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  if (warp == 0 || warp == 2) {
    // ------------------------------------------------ keys (0) and values (2)
    const bool is_k = warp == 0;
    constexpr int KEYS_K = 64, KEYS_V = 128;
    const uint32_t ring = sm + (is_k ? C::OFF_K : C::OFF_V);
    int sent = 0;  // tiles whose copies have been issued
    // the barrier that K(j) or V(j) is announced on, and the wait for its stage
    auto full_bar = [&](int j) {
      return is_k && j < C::NS ? B.k_first(j) : B.ready(j % C::NS);
    };
    // (V(j), j < NS, waits for Q K(j) although its stage is empty: a parity names a
    // phase only to who has seen the one before)
    auto stage_free = [&](int j) -> bool {
      if (is_k && j < C::NS) return true;
      return warp_wait(B.moved(j % C::NS), (is_k ? (j / C::NS) - 1 : j / C::NS) & 1, abort_flag, p.err);
    };
    const uint16_t* base = is_k ? p.c.k + h * p.c.head_stride
                                : p.c.v + h * p.c.head_stride + rank * (D / 2);
    // rows [i0, i0 + 32) of a stage by 16-byte copies, lane l's row at element
    // offset `off` (-1: zeros)
    auto copy32_k = [&](uint32_t dst, int i0, long long off) {
      constexpr int CH = D / 8, RPI = 32 / CH;  // pieces of a key; keys a warp copies at once
#pragma unroll 8
      for (int i = 0; i < 32 / RPI; ++i) {
        const int r = i0 + i * RPI + lane / CH, c = lane % CH;
        const long long o = __shfl_sync(0xffffffffu, off, r & 31);
        cp_async16(dst + (c >> 3) * (KEYS_K * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                   base + (o >= 0 ? o : 0) + c * 8, o >= 0 ? 16u : 0u);
      }
    };
    // rows [i0, i0 + count), offsets held by the lanes of row modulo 32
    auto copy_v = [&](uint32_t dst, int i0, int count, long long off) {
      constexpr int CH = D / 16, RPI = 32 / CH;  // pieces of half a value
      for (int i = 0; i < count / RPI; ++i) {
        const int r = i0 + i * RPI + lane / CH, c = lane % CH;
        const long long o = __shfl_sync(0xffffffffu, off, r & 31);
        const uint32_t at = D == 64 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4)
                                    : (c >> 3) * (KEYS_V * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
        cp_async16(dst + at, base + (o >= 0 ? o : 0) + c * 8, o >= 0 ? 16u : 0u);
      }
    };
    if constexpr (TMA) {
      // At most one box a lane: box `y` of the stage's rows, `x` of its features.
      // A lane's page number is looked up a tile ahead.
      constexpr int FW = (D == 64) ? 32 : 64;       // features of a box of V
      const int box = 1 << cp.box_log2;
      const int fc_log2 = is_k ? (D == 256 ? 2 : (D == 128 ? 1 : 0)) : (D == 256 ? 1 : 0);
      const int x = lane & ((1 << fc_log2) - 1), y = lane >> fc_log2;
      const int stage_rows = is_k ? KEYS_K : KEYS_V;
      const bool mine = (y << cp.box_log2) < stage_rows;
      const int row0 = (is_k ? rank * KEYS_K : 0) + (y << cp.box_log2);  // first row in the tile
      const uint32_t at = is_k ? x * (KEYS_K * 128) + (y << cp.box_log2) * 128
                               : x * (KEYS_V * 128) + (y << cp.box_log2) * FW * 2;
      const int feature = is_k ? x * 64 : rank * (D / 2) + x * FW;
      int page_row = 0, page = 0;
      auto look = [&](int j) {
        const int key = first + j * kTileKeys + row0;
        if (mine && j < nb && key < hi) {
          const int col = fast_div(key, p.c.div);
          page_row = key - col * p.c.page;
          page = table[col];
        }
      };
      look(0);
      for (int j = 0; j < nb; ++j) {
        const uint32_t bar = full_bar(j), full = mapa_shared(bar, 0);
        const uint32_t dst = ring + (j % C::NS) * C::STAGE;
        const int t0 = first + j * kTileKeys;
        // rows of the tile that hold keys of the chunk, [e0, e1), and the boxes
        // that are loaded: all with such a row (K); those with no other row (V)
        const int e0 = max(lo - t0, 0), e1 = min(hi - t0, kTileKeys);
        const int up = is_k ? 0 : box - 1, dn = is_k ? box - 1 : 0;
        const int w0 = (e0 + up) & ~(box - 1), w1 = (e1 + dn) & ~(box - 1);
        if (!stage_free(j)) break;
        if (rank == 0 && lane == 0) {
          const uint32_t bytes = (uint32_t)max(w1 - w0, 0) * D * 2;  // both CTAs'
          asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes)
                       : "memory");
        }
        if (mine && row0 >= w0 && row0 < w1)
          tma_box_pair(dst + at, is_k ? &cp.k : &cp.v, feature, page_row, h,
                       (page < 0 || page > p.c.pages) ? p.c.pages : page, full);
        sent = j + 1;
        look(j + 1);
        bool copied = false;
        if (!is_k && (e0 > 0 || w1 < kTileKeys)) {
          // the edges of the chunk: what the product's 16-key steps touch besides
          const int end = (e1 + 15) & ~15;
          for (int i0 = e0 & ~15; i0 < end; i0 += 8) {
            if (i0 >= w0 && i0 < w1) continue;
            const int key = t0 + (i0 & ~31) + lane;
            copy_v(dst, i0, 8, key >= lo ? lookup(key) : -1);
            copied = true;
          }
          if (copied) {
            cp_async_commit();
            cp_async_wait<0>();
            fence_proxy_async_smem();
          }
        }
        __syncwarp();
        if (lane == 0) {
          if (copied) arrive_release_cluster(full);
          else mbar_arrive_cluster(full);
        }
      }
    } else {
      for (int j = 0; j < nb; ++j) {
        const uint32_t dst = ring + (j % C::NS) * C::STAGE;
        const int t0 = first + j * kTileKeys;
        if (!stage_free(j)) break;
        sent = j + 1;
#pragma unroll
        for (int i0 = 0; i0 < KEYS_V; i0 += 32) {
          if (is_k && i0 >= KEYS_K) break;
          const long long off = lookup(t0 + (is_k ? rank * KEYS_K : 0) + i0 + lane);
          if (is_k) copy32_k(dst, i0, off);
          else copy_v(dst, i0, 32, off);
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_release_cluster(mapa_shared(full_bar(j), 0));
      }
    }
    cp_async_wait<0>();
    // No CTA leaves while a copy of the pair is in flight (in the usual course
    // the products have waited for all of them; after a wait has given up
    // nothing has): the even CTA's barriers count the bytes of both.
    if (rank == 0) {
      for (int j = max(sent - C::NS, 0); j < sent; ++j)
        copies_done(full_bar(j), is_k ? (j < C::NS ? 0 : ((j / C::NS) - 1) & 1) : (j / C::NS) & 1);
    }
    // The last tiles have no K(j + NS) to wait for.  (After the wait above, which
    // these arrivals' phases could otherwise overtake.)
    if (is_k && sent == nb) {
      for (int j = max(nb, C::NS); j < nb + C::NS; ++j) {
        if (!stage_free(j)) break;
        if (lane == 0) mbar_arrive_cluster(mapa_shared(full_bar(j), 0));
      }
    }
  } else {
    // ---------------------------------------------------------- MMA issuer
    const int nb_all = nb, lo_all = lo, hi_all = hi, first_all = first;
    const uint32_t tmem_all = tmem, sm_all = sm;
    // One warp issues everything, in the order P V(j), Q K(j + NS): P(j) gives
    // way to the scores of tile j + NS without a wait, since the tensor core
    // takes a thread's MMAs in the order of issue.  (Two warps, one for each
    // product, had their MMAs interleaved and both finished late.)
    if (rank == 0 && warp == 1) {
      // broadcast, so that the compiler knows them to be the same in all lanes and
      // keeps operands and counters in uniform registers, which the MMAs take
      const int nb = __shfl_sync(0xffffffffu, nb_all, 0), lo = __shfl_sync(0xffffffffu, lo_all, 0);
      const int hi = __shfl_sync(0xffffffffu, hi_all, 0), first = __shfl_sync(0xffffffffu, first_all, 0);
      const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_all, 0), sm = __shfl_sync(0xffffffffu, sm_all, 0);
      const Bars<D> B{sm + C::OFF_BAR};
      const uint32_t id_qk = idesc_f16(256, kTileKeys, BF ? 1 : 0);
      const uint32_t id_pv = idesc_f16(256, D, BF ? 1 : 0) | (1u << 16);  // B: N contiguous
      const uint64_t aq = sdesc_k_sw128(sm);
      const uint64_t bk0 = sdesc_k_sw128(sm + C::OFF_K);
      const uint64_t bv0 = D == 64 ? sdesc_mn(sm + C::OFF_V, 64, 0)
                                   : sdesc_mn(sm + C::OFF_V, 128, 128 * 128);
      constexpr int STEP = (D == 64 ? 16 * 64 : 16 * 128) / 16;  // descriptor units of 16 keys
      auto qk = [&](int s) {
#pragma unroll
        for (int kk = 0; kk < D / 64; ++kk)
          mma_ss_x4(tmem + C::S_COL + s * 128, aq + kk * (128 * 128 / 16),
                    bk0 + s * (C::STAGE / 16) + kk * (64 * 128 / 16), id_qk, kk ? 1u : 0u);
      };
      bool ok = warp_wait<true>(B.q_full(), 0, abort_flag, p.err);
      for (int t = 0; ok && t < min(C::NS, nb); ++t) {
        ok = warp_wait<!TMA>(B.k_first(t), 0, abort_flag, p.err);
        tc_fence_after();
        if (ok) {
          qk(t);
          tc_commit_pair_mc_w(B.moved(t), 3);
        }
      }
      int s = 0;
      uint32_t par = 0;
      for (int j = 0; ok && j < nb; ++j) {
        const int t0 = first + j * kTileKeys;
        const bool inner = t0 >= lo && t0 + kTileKeys <= hi;  // not at the chunk's edges
        if (!((TMA && inner) ? warp_wait(B.ready(s), par, abort_flag, p.err)
                             : warp_wait<true>(B.ready(s), par, abort_flag, p.err)))
          break;
        tc_fence_after();
        const uint32_t a = tmem + C::S_COL + s * 128;
        const uint64_t b = bv0 + s * (C::STAGE / 16);
        if (inner) {
          mma_ts_x4<STEP>(tmem, a, b, id_pv, j > 0 ? 1u : 0u);
          mma_ts_x4<STEP>(tmem, a + 32, b + 4 * STEP, id_pv, 1u);
        } else {
          // the 16-key steps that hold a key of the chunk
          const int ka = max(lo - t0, 0) >> 4, kz = (min(hi - t0, kTileKeys) + 15) >> 4;
          for (int kk = ka; kk < kz; ++kk)
            tc_mma_f16_ts_pair_w(tmem, a + 8 * kk, b + STEP * kk, id_pv, (j > 0 || kk > ka) ? 1u : 0u);
        }
        if (j + C::NS < nb) qk(s);
        tc_commit_pair_mc_w(B.moved(s), 3);
        if (++s == C::NS) {
          s = 0;
          par ^= 1;
        }
      }
      tc_commit_pair_mc_w(B.drain(), 3);
    }
    // every MMA has finished before TMEM is released
    if (warp == 1 && lane == 0) mbar_wait_bounded(B.drain(), 0, abort_flag, kWaitLimitNs);
  }
  } else {
    // ------------------------------------------- softmax, correction, epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    bool any_bad;
    {
      // Q: warp w copies rows 8 w .. 8 w + 7 of the CTA's 128
      constexpr int CH = D / 8, RPI = 32 / CH;
#pragma unroll 4
      for (int i = 0; i < 8 / RPI; ++i) {
        const int r = (warp - kSoftWarp0) * 8 + i * RPI + lane / CH, c = lane % CH;
        const int gr = r0 + rank * 128 + r;
        const bool in = gr < r1;
        const int tk = in ? fast_div(gr, p.divG) : 0;
        const uint16_t* src =
            p.q + (in ? (s.t0 + tk) * p.q_ts + (h * p.G + gr - tk * p.G) * p.q_hs : 0) + c * 8;
        cp_async16(sm + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4), src,
                   in ? 16u : 0u);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_release_cluster(mapa_shared(B.q_full(), 0));
      // page numbers of this chunk that are bad (then every score is looked at)
      int bad = 0;
      for (int i = fast_div(lo, p.c.div) + threadIdx.x - 32 * kSoftWarp0;
           i <= fast_div(hi - 1, p.c.div); i += 32 * kSoftWarps) {
        const int pg = table[i];
        if (pg < 0 || pg >= p.c.pages) bad = 1;
      }
      any_bad = softmax_any(bad);
      if (any_bad && threadIdx.x == 32 * kSoftWarp0) atomicOr(p.err, PAGED_DEVERR_PAGE);
    }
    // visible keys of the row: [vlo, vhi); rows that do not exist see all (of zeros)
    int vlo = 0, vhi = 0x7fffffff;
    if (valid) {
      const int pos = s.kv - s.nq + tok;
      vhi = p.causal || pos < 0 ? min(s.kv, pos + 1) : s.kv;
      vlo = p.window > 0 ? window_begin(pos, p.window) : 0;
    } else {
      vhi = s.kv;
    }
    vlo = max(vlo, lo);
    int wlo = vlo, whi = vhi;  // the warp's strictest bounds
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      wlo = max(wlo, __shfl_xor_sync(0xffffffffu, wlo, d));
      whi = min(whi, __shfl_xor_sync(0xffffffffu, whi, d));
    }
    // sh_ref [4][128]: a row's reference maximum after tile j, in slot j & 3;
    // sh_max [slot][half][128]: the halves' maxima of a tile, slot j & 3
    float* sh_ref = reinterpret_cast<float*>(smem + C::OFF_REF);
    float* sh_max = reinterpret_cast<float*>(smem + C::OFF_MAX);
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t ready0 = mapa_shared(B.ready(0), 0);
    const float c = p.scale_log2;
    // the reference that this thread's sum l (over its own scores) is relative to
    float m = kNegInf, l = 0.f;
    // The weights are rounded to 16 bits for the product, l sums them unrounded
    // (the lse is its logarithm).  With a lagging reference the largest weight,
    // which the result follows most, is rounded like any other; so the result is
    // divided by l with the rounding of each tile's largest weight put back:
    // `extra` is what that adds up to (of the row: in one half's threads).
    float extra = 0.f;
    if (group == 1 && half == 0) {  // "after tile -1"
      sh_ref[3 * 128 + trow] = kNegInf;
      tile_arrive(0, quarter);
    }
    // after a wait has given up, the warp runs on without waiting (others may
    // stand at a common barrier) and writes no result
    bool ok = true;
    bool far = false;  // some row of the warp has a reference past kFar
    for (int j = group; j < nb; j += 2) {
      const int sb = j % C::NS;
      ok = ok && warp_wait(B.moved(sb), (j / C::NS) & 1, abort_flag, p.err);
      tc_fence_after();
      const uint32_t ts = tmem + lanes + C::S_COL + sb * 128;
      uint32_t x[2][32];
      tmem_ld32(ts + half * 64, x[0]);
      tmem_ld32(ts + half * 64 + 32, x[1]);
      tmem_ld_wait();
      const int k0 = first + j * kTileKeys + half * 64;
      if (k0 < wlo || k0 + 64 > min(whi, hi) || any_bad) {
        const int a = vlo - k0, z = min(vhi, hi) - k0;  // visible: a <= i < z
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (i < a || i >= z) x[i >> 5][i & 31] = __float_as_uint(kNegInf);
        if (any_bad) {  // rare: the page numbers are looked at again
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t out = 0;
#pragma unroll 1
            for (int i = max(a - 32 * q, 0); i < min(z - 32 * q, 32); ++i)
              if (lookup(k0 + 32 * q + i) < 0) out |= 1u << i;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (out >> i & 1) x[q][i] = __float_as_uint(kNegInf);
          }
        }
      }
      float mt[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t* y = x[e >> 1] + (e & 1) * 16;
        mt[e] = __uint_as_float(y[0]);
#pragma unroll
        for (int i = 1; i < 15; i += 2)
          mt[e] = max3(mt[e], __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
        mt[e] = fmaxf(mt[e], __uint_as_float(y[15]));
      }
      float mx = fmaxf(max3(mt[0], mt[1], mt[2]), mt[3]);
      // one barrier for the halves' maxima, for the reference after the tile
      // before, and for P to replace scores that the other half has read
      sh_max[((j & 3) * 2 + half) * 128 + trow] = mx;
      tile_wait(group, quarter);
      mx = fmaxf(mx, sh_max[((j & 3) * 2 + (half ^ 1)) * 128 + trow]);
      const float ref = sh_ref[((j - 1) & 3) * 128 + trow];
      const bool rise = (mx - ref) * c > kRise || (ref == kNegInf && mx > ref);
      const float now = rise ? mx : ref;
      if (half == 0) {
        sh_ref[(j & 3) * 128 + trow] = now;
        if (j + 1 < nb) tile_arrive(group ^ 1, quarter);
      }
      if (__any_sync(0xffffffffu, now != m)) {
        if (j > 0 && __any_sync(0xffffffffu, rise)) {
          // P V of the tiles before has been added up before O changes
          ok = ok && warp_wait(B.moved((j - 1) % C::NS), ((j - 1) / C::NS + 1) & 1, abort_flag, p.err);
          tc_fence_after();
          const float f = rise ? ex2((ref - now) * c) : 1.f;
#pragma unroll 1
          for (int f0 = 0; f0 < D / 2; f0 += 16) {
            uint32_t o[16];
            const uint32_t to = tmem + lanes + half * (D / 2) + f0;
            tmem_ld16(to, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(to, o);
          }
          tmem_st_wait();
        }
        const float f = m == kNegInf ? 0.f : ex2((m - now) * c);
        l *= f;
        extra *= f;
        m = now;
        far = __any_sync(0xffffffffu, m != kNegInf && fabsf(m * c) > kFar);
      }
      float mc = m == kNegInf ? 0.f : fmaf(m, c, -kShift<BF>);
      if (far) {
        const float s = m == kNegInf ? 0.f : m;
#pragma unroll
        for (int i = 0; i < 64; ++i)
          x[i >> 5][i & 31] = __float_as_uint(__uint_as_float(x[i >> 5][i & 31]) - s);
        mx -= s;
        mc = -kShift<BF>;
      }
      {
        const float top = ex2(fmaf(mx, c, -mc));
        extra += round16<BF>(top) - top;
      }
      // two values at a time where the machine can: x c - mc, and the sums
      const uint64_t c2 = pack_f2(c, c), mc2 = pack_f2(-mc, -mc);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint64_t t = fma_f2(pack_u2(x[q][2 * i], x[q][2 * i + 1]), c2, mc2);
          float e0, e1;
          unpack_f2(t, e0, e1);
          e0 = ex2(e0);
          e1 = ex2(e1);
          sum[i & 1] = add_f2(sum[i & 1], pack_f2(e0, e1));
          pk[i] = pack2<BF>(e0, e1);
        }
        tmem_st16(ts + half * 32 + 16 * q, pk);
      }
      {
        float a0, a1;
        unpack_f2(add_f2(sum[0], sum[1]), a0, a1);
        l += a0 + a1;
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      // (what this arrival publishes lies in TMEM, ordered by the tcgen05 fences;
      // a release at cluster scope here costs several hundred cycles a tile)
      if (lane == 0) mbar_arrive_cluster(ready0 + 8 * sb);
    }
    // ---- epilogue: a quarter of the features each
    ok = ok && warp_wait(B.drain(), 0, abort_flag, p.err);
    // the row's whole sum from its four parts
    const int part = half + 2 * group;
    float4* sh_ml = reinterpret_cast<float4*>(smem + C::OFF_ML);
    sh_ml[part * 128 + trow] = make_float4(m, l, half == 0 ? extra : 0.f, 0.f);
    quarter_sync(quarter);
    {
      float top = kNegInf;  // the last tile's reference, O's
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, sh_ml[i * 128 + trow].x);
      l = extra = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 y = sh_ml[i * 128 + trow];
        // (no key seen: (-inf) - (-inf); there l is 0, or NaN where the scores were,
        // which raise no maximum)
        const float f = y.x == top ? 1.f : ex2((y.x - top) * c);
        l += y.y * f;
        extra += y.z * f;
      }
      m = top;
    }
    if (ok) {
      tc_fence_after();
      // (a part of a row: for a join that divides by the sum of the l)
      const float inv = l == 0.f ? 0.f : (p.chunks > 1 ? l : 1.f) / (l + extra);
      const float mlog = fmaf(m, c, -kShift<BF>);  // (-inf: no key seen)
#pragma unroll 1
      for (int f0 = 0; f0 < D / 4; f0 += 16) {
        const int f = part * (D / 4) + f0;
        uint32_t o[16];
        tmem_ld16(tmem + lanes + f, o);
        tmem_ld_wait();
        if (!valid) continue;
        if (p.chunks > 1) {
          float4* d4 = reinterpret_cast<float4*>(p.part_o + (rid * p.chunks + ck) * D + f);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            d4[i] = make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv,
                                __uint_as_float(o[4 * i + 2]) * inv, __uint_as_float(o[4 * i + 3]) * inv);
        } else {
          uint16_t* dst = p.o + (s.t0 + tok) * p.o_ts + head * p.o_hs + f;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint4 v;
            v.x = pack2<BF>(__uint_as_float(o[8 * i]) * inv, __uint_as_float(o[8 * i + 1]) * inv);
            v.y = pack2<BF>(__uint_as_float(o[8 * i + 2]) * inv, __uint_as_float(o[8 * i + 3]) * inv);
            v.z = pack2<BF>(__uint_as_float(o[8 * i + 4]) * inv, __uint_as_float(o[8 * i + 5]) * inv);
            v.w = pack2<BF>(__uint_as_float(o[8 * i + 6]) * inv, __uint_as_float(o[8 * i + 7]) * inv);
            reinterpret_cast<uint4*>(dst)[i] = v;
          }
        }
      }
      if (valid && part == 0) {
        if (p.chunks > 1) p.part_ml[rid * p.chunks + ck] = make_float2(mlog, l);
        else if (p.lse) p.lse[rid] = l == 0.f ? kNegInf : kLn2 * mlog + logf(l);
      }
    }
  }

  leave();
}

template <int D, bool BF, bool TMA>
cudaError_t chunk_launch_t(const ChunkParams& cp, cudaStream_t st) {
  using C = ChunkCfg<D>;
  const AttnParams& p = cp.a;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem((const void*)paged_chunk_kernel<D, BF, TMA>, C::SMEM, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(2ll * p.tiles * p.c.heads * p.chunks));
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = C::SMEM;
  c.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = 2;
  a[0].val.clusterDim.y = 1;
  a[0].val.clusterDim.z = 1;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, paged_chunk_kernel<D, BF, TMA>, cp);
}

template <int D, bool BF>
cudaError_t chunk_launch(const AttnParams& p, cudaStream_t st) {
  ChunkParams cp;
  cp.a = p;
  int box = 64;
  cp.box_log2 = 6;
  while (p.c.page % box) {
    box >>= 1;
    --cp.box_log2;
  }
  if (box >= 8 && make_page_map(&cp.k, p.c.k, p.c, 64, box, BF) &&
      make_page_map(&cp.v, p.c.v, p.c, D == 64 ? 32 : 64, box, BF))
    return chunk_launch_t<D, BF, true>(cp, st);
  return chunk_launch_t<D, BF, false>(cp, st);
}

}  // namespace

cudaError_t launch_paged_chunk(const AttnParams& p, bool bf16, cudaStream_t st) {
  switch (p.c.dim) {
    case 64: return bf16 ? chunk_launch<64, true>(p, st) : chunk_launch<64, false>(p, st);
    case 128: return bf16 ? chunk_launch<128, true>(p, st) : chunk_launch<128, false>(p, st);
    case 256: return bf16 ? chunk_launch<256, true>(p, st) : chunk_launch<256, false>(p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
