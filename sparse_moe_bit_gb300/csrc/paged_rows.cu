// Attention of a few query rows of a key/value head over the paged cache, and
// the join of results that were split over the keys (include/paged.h).
//
// The G query heads that share a key/value head and the sequence's new tokens
// form the rows of one small matrix: row r is token r / G, head r % G of the
// group.  A CTA takes 16 rows (one mma tile) of a sequence and a chunk of its
// keys, so that every key and value is read from HBM once for the whole group.
//   S = Q K^T, m' = max(m, rowmax S), P = 2^(S - m'), l = l 2^(m - m') + sum P,
//   O = O 2^(m - m') + P V                         (S in log2 units, all fp32)
//
// Bound: HBM (2 bytes x 2 D per key against 2 x 4 D x rows operations).  What
// counts is bytes in flight, so each of the four warps streams keys of its own
// (groups of 16, dealt round robin) through a ring of its own, filled by
// 16-byte asynchronous copies two groups ahead, with its own m, l and O: the
// warps meet once, at the end.  The product of 16 rows by mma.sync
// (m16n8k16) needs a tenth of the rate at which keys arrive; wider row tiles
// go to the tcgen05 kernel.  Page numbers of a warp's next group are fetched a
// group before its copies are issued.  Rows of a page that lie behind the
// sequence's end, or whose page number is bad, are never read: the copy fills
// them with zeros and the score is masked.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kGroup = 16;  // keys of a warp's step

template <int D>
struct RowsCfg {
  static constexpr int ROW = 2 * D;  // bytes of a key
  static constexpr int STAGES = D == 64 ? 4 : 3;
  static constexpr int STAGE = 2 * kGroup * ROW;  // keys and values of a group
  static constexpr int RING = kWarps * STAGES * STAGE;
  static constexpr int OFF_Q = RING;
  static constexpr int SMEM = RING + kRowTile * ROW;
  static_assert(kWarps * kRowTile * D * 4 <= RING, "the warps' results fit the ring");
};

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

template <int D, bool BF>
__global__ void __launch_bounds__(32 * kWarps) paged_rows_kernel(const AttnParams p) {
  using C = RowsCfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sh_m[kWarps][kRowTile], sh_l[kWarps][kRowTile];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the join, if there is one, may be set up while this grid runs
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  int bid = blockIdx.x;
  const int ck = bid % p.chunks;
  bid /= p.chunks;
  const int h = bid % p.c.heads;
  bid /= p.c.heads;
  const int tile0 = bid % p.tiles;
  const int n = bid / p.tiles;
  const Seq s = load_seq(p.b, n);
  const int rows = s.nq * p.G;
  const int32_t* table = p.b.table + n * p.b.table_stride;
  const uint16_t* kbase = p.c.k + h * p.c.head_stride;
  const uint16_t* vbase = p.c.v + h * p.c.head_stride;
  const uint32_t sm = smem_u32(smem);
  const uint32_t qs = sm + C::OFF_Q;
  const uint32_t ring = sm + warp * C::STAGES * C::STAGE;

  for (int tile = tile0; tile * kRowTile < rows; tile += p.tiles) {
    const int r0 = tile * kRowTile, r1 = min(r0 + kRowTile, rows);
    const int2 kr = key_range(p, s, r0, r1);
    const int span = kr.y - kr.x;
    // keys of this chunk
    const long long c0 = (long long)ck * p.chunk;
    const int lo = kr.x + (int)min(c0, (long long)span);
    const int hi = ck == p.chunks - 1 ? kr.y : kr.x + (int)min(c0 + p.chunk, (long long)span);
    const int groups = (hi - lo + kGroup - 1) / kGroup;
    const int steps = groups > warp ? (groups - warp + kWarps - 1) / kWarps : 0;

    // ---- Q rows into shared memory, 16-byte chunks swizzled by the row
    for (int i = threadIdx.x; i < kRowTile * (C::ROW / 16); i += 32 * kWarps) {
      const int r = i / (C::ROW / 16), c = i % (C::ROW / 16);
      const bool ok = r0 + r < r1;
      const int tok = ok ? fast_div(r0 + r, p.divG) : 0;
      const int g = ok ? r0 + r - tok * p.G : 0;
      const uint16_t* src =
          p.q + (ok ? (long long)(s.t0 + tok) * p.q_ts + (long long)(h * p.G + g) * p.q_hs : 0);
      cp_async16(qs + r * C::ROW + ((c ^ (r & 7)) << 4), src + c * 8, ok ? 16u : 0u);
    }
    cp_async_commit();

    // ---- the ring: lane l (and l + 16) addresses key l of a group
    auto lookup = [&](int st) -> long long {  // element offset of the lane's key; -1: none
      const int key = lo + (warp + st * kWarps) * kGroup + (lane & 15);
      if (st >= steps || key >= hi) return -1;
      const int col = fast_div(key, p.c.div);
      const int pg = table[col];
      if (pg < 0 || pg >= p.c.pages) {
        if (lane < 16) atomicOr(p.err, PAGED_DEVERR_PAGE);
        return -1;
      }
      return pg * p.c.page_stride + (key - col * p.c.page) * p.c.row_stride;
    };
    auto issue = [&](int st, long long off) {
      if (st < steps) {
        const uint32_t kd = ring + (st % C::STAGES) * C::STAGE, vd = kd + kGroup * C::ROW;
        constexpr int CH = C::ROW / 16;     // 16-byte chunks of a key
        constexpr int RPI = 32 / CH > 0 ? 32 / CH : 1;  // keys a warp copies at once
#pragma unroll
        for (int i = 0; i < kGroup / RPI; ++i) {
          const int r = i * RPI + lane / CH, c = lane % CH;
          const long long o = __shfl_sync(0xffffffffu, off, r);
          const uint32_t nb = o >= 0 ? 16u : 0u;
          const long long e = (o >= 0 ? o : 0) + c * 8;
          const uint32_t d = r * C::ROW + ((c ^ (r & 7)) << 4);
          cp_async16(kd + d, kbase + e, nb);
          cp_async16(vd + d, vbase + e, nb);
        }
      }
      cp_async_commit();
    };
    uint32_t seen[C::STAGES];  // per stage: the group's keys that may be scored
    long long off = lookup(0);
#pragma unroll
    for (int st = 0; st < C::STAGES - 1; ++st) {
      seen[st] = __ballot_sync(0xffffffffu, off >= 0) & 0xffffu;
      issue(st, off);
      off = lookup(st + 1);
    }
    cp_async_wait<C::STAGES - 1>();  // Q
    __syncthreads();

    // per-thread rows: g and g + 8 of the tile
    const int g = lane >> 2, t2 = (lane & 3) * 2;
    int hiA, hiB, loA, loB;  // visible keys of the two rows: [lo, hi)
    {
      auto range = [&](int r, int& a, int& b) {
        const int pos = s.kv - s.nq + fast_div(min(r0 + r, rows - 1), p.divG);
        b = p.causal ? min(s.kv, pos + 1) : s.kv;
        a = p.window > 0 ? pos - p.window + 1 : 0;
      };
      range(g, loA, hiA);
      range(g + 8, loB, hiB);
    }
    float mA = kNegInf, mB = kNegInf, lA = 0.f, lB = 0.f;
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;

    const int mi = lane >> 3, mr = lane & 7;  // ldmatrix: matrix and row of this lane
#pragma unroll 1
    for (int s0 = 0; s0 < steps; s0 += C::STAGES) {
#pragma unroll
      for (int ss = 0; ss < C::STAGES; ++ss) {
        const int st = s0 + ss;
        if (st >= steps) break;
        // the next group's copies go to the stage read one step ago
        {
          constexpr int A = C::STAGES - 1;
          const int nx = (ss + A) % C::STAGES;
          seen[nx] = __ballot_sync(0xffffffffu, off >= 0) & 0xffffu;
          issue(st + A, off);
          off = lookup(st + A + 1);
        }
        cp_async_wait<C::STAGES - 1>();
        __syncwarp();
        const uint32_t ks = ring + ss * C::STAGE, vs = ks + kGroup * C::ROW;
        // S: two blocks of 8 keys, two accumulators each to halve the chains
        float sc[2][2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[i][j][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t a[4], b[4];
          // A: matrices (rows 0-7, k 0-7), (rows 8-15, k 0-7), (0-7, 8-15), (8-15, 8-15)
          {
            const int r = (mi & 1) * 8 + mr, c = 2 * kk + (mi >> 1);
            ldsm4(a, qs + r * C::ROW + ((c ^ (r & 7)) << 4));
          }
          {
            const int r = (mi >> 1) * 8 + mr, c = 2 * kk + (mi & 1);
            ldsm4(b, ks + r * C::ROW + ((c ^ (r & 7)) << 4));
          }
          mma16816<BF>(sc[0][kk & 1], a, b[0], b[1]);
          mma16816<BF>(sc[1][kk & 1], a, b[2], b[3]);
        }
        const int key0 = lo + (warp + st * kWarps) * kGroup;
        const uint32_t ok = seen[ss];
        float x[2][4];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int kx = nb * 8 + t2 + (e & 1);
            const int key = key0 + kx;
            const bool vis = (ok >> kx & 1) && (e < 2 ? (key >= loA && key < hiA)
                                                      : (key >= loB && key < hiB));
            x[nb][e] = vis ? (sc[nb][0][e] + sc[nb][1][e]) * p.scale_log2 : kNegInf;
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
          ldsm4t(b, vs + r * C::ROW + ((c ^ (r & 7)) << 4));
          mma16816<BF>(o[2 * nn], pa, b[0], b[1]);
          mma16816<BF>(o[2 * nn + 1], pa, b[2], b[3]);
        }
        __syncwarp();  // the stage is read before the next step's copies overwrite it
      }
    }
    cp_async_wait<0>();
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
      lA += __shfl_xor_sync(0xffffffffu, lA, d);
      lB += __shfl_xor_sync(0xffffffffu, lB, d);
    }
    // ---- the four warps' results, joined in warp order
    __syncthreads();  // every warp is done with the ring
    float* so = reinterpret_cast<float*>(smem);  // [warp][row][D]
    {
      float* w = so + warp * kRowTile * D;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        *reinterpret_cast<float2*>(w + g * D + i * 8 + t2) = make_float2(o[i][0], o[i][1]);
        *reinterpret_cast<float2*>(w + (g + 8) * D + i * 8 + t2) = make_float2(o[i][2], o[i][3]);
      }
      if ((lane & 3) == 0) {
        sh_m[warp][g] = mA;
        sh_m[warp][g + 8] = mB;
        sh_l[warp][g] = lA;
        sh_l[warp][g + 8] = lB;
      }
    }
    __syncthreads();
    constexpr int PER = D / 8;  // 8 features a thread
    for (int i = threadIdx.x; i < (r1 - r0) * PER; i += 32 * kWarps) {
      const int r = i / PER, f = (i % PER) * 8;
      float m = kNegInf;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sh_m[w][r]);
      const float u = m == kNegInf ? 0.f : m;
      float l = 0.f, acc[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float a = exp2_approx(sh_m[w][r] - u);
        l += a * sh_l[w][r];
        const float4* q4 = reinterpret_cast<const float4*>(so + (w * kRowTile + r) * D + f);
        const float4 y = q4[0], z = q4[1];
        acc[0] += a * y.x;
        acc[1] += a * y.y;
        acc[2] += a * y.z;
        acc[3] += a * y.w;
        acc[4] += a * z.x;
        acc[5] += a * z.y;
        acc[6] += a * z.z;
        acc[7] += a * z.w;
      }
      const int tok = fast_div(r0 + r, p.divG);
      const int head = h * p.G + (r0 + r - tok * p.G);
      const long long rid = (long long)(s.t0 + tok) * p.Hq + head;
      if (p.chunks > 1) {
        const long long at = rid * p.chunks + ck;
        float4* d4 = reinterpret_cast<float4*>(p.part_o + at * D + f);
        d4[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        d4[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (f == 0) p.part_ml[at] = make_float2(m, l);
      } else {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint4 v;
        v.x = pack2<BF>(acc[0] * inv, acc[1] * inv);
        v.y = pack2<BF>(acc[2] * inv, acc[3] * inv);
        v.z = pack2<BF>(acc[4] * inv, acc[5] * inv);
        v.w = pack2<BF>(acc[6] * inv, acc[7] * inv);
        *reinterpret_cast<uint4*>(p.o + (s.t0 + tok) * p.o_ts + head * p.o_hs + f) = v;
        if (f == 0 && p.lse) p.lse[rid] = l == 0.f ? kNegInf : kLn2 * m + logf(l);
      }
    }
    __syncthreads();  // sh_* and the ring are read before the next tile
  }
}

// Join of a row's chunks, in chunk order: warp w of the row's CTA takes chunks
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
  const float2* ml = p.part_ml + rid * p.chunks;
  float m = kNegInf;
  for (int c = lane; c < p.chunks; c += 32) m = fmaxf(m, ml[c].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float u = m == kNegInf ? 0.f : m;
  float l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  const float* po = p.part_o + rid * p.chunks * D;
#pragma unroll 4
  for (int c = warp; c < p.chunks; c += W) {
    const float2 x = ml[c];
    const float a = exp2_approx(x.x - u);
    l += a * x.y;
    if (x.y != 0.f) {  // (an empty chunk wrote zeros; NaN sums pass)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += a * po[(long long)c * D + e * 32 + lane];
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

template <int D, bool BF>
cudaError_t rows_launch(const AttnParams& p, cudaStream_t st) {
  using C = RowsCfg<D>;
  static bool attr_set = false;
  if (!attr_set) {
    const cudaError_t e = cudaFuncSetAttribute(
        paged_rows_kernel<D, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_set = true;
  }
  const long long grid = (long long)p.b.N * p.tiles * p.c.heads * p.chunks;
  return launch_kernel(paged_rows_kernel<D, BF>, dim3((unsigned)grid), dim3(32 * kWarps), C::SMEM,
                       st, p);
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
  // a warp per eight chunks, so that a long split is not read by one warp alone
  if (p.chunks > 16) return join_w<D, BF, 8>(p, st);
  return join_w<D, BF, 2>(p, st);
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
