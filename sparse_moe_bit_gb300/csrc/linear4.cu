// Products of a few tokens with 4-bit weights in the checkpoint's layout
// (include/step.h).
//
//   y[t][o] = sum over groups of (s sum c x + b sum x)
// so the products of a group run on the codes themselves, which are exact in 16 bits,
// and scale and bias enter once a group in fp32:
//   bf16:  a code with the exponent of 128 in front is 128 + c (8 significant bits), and
//          the group's sum is s (acc - 128 X) + b X with X = sum x
//   fp16 (8-bit x too, which fp16 holds exactly):  a code's bits alone are the subnormal
//          c 2^-24, and the group's sum is (2^24 s) acc + b X
// An 8-bit x has its own scale applied after a 64-wide part (or at the end, where a
// token has one).
//
// Bound: HBM (half a byte a weight plus four a group).  A warp has 16 rows of weights as
// the wide side of mma.sync (m16n8k16) and 8 NT tokens as the narrow one, so that up to
// 64 tokens share one reading.  Lane (g, j) of a warp holds rows g and g + 8 and in each
// part of 64 weights the codes 16 j .. 16 j + 15: 8 bytes a row, four lanes a sector, which
// the shifts turn into operands in the order 0 4 1 5 2 6 3 7; the tokens are laid out in
// shared memory in that order once.  Loads go straight to registers, four parts ahead
// (2.3 KB a warp), across blocks of rows, so that a CTA that walks many never drains.
//
// Split: a CTA holds WR row tiles x WK slices of K (WR WK = 8 warps), and a cluster of C
// CTAs splits K again where there are few rows or the tokens of all of K do not fit
// shared memory; partial sums meet in shared memory, in the order of K.
#include "paged_internal.h"
#include "ptx.cuh"
#include "step_internal.h"

namespace moe {
namespace {

constexpr int kWarps = 8;

struct Plan4 {
  Linear4Params a;
  int wr, wk, cluster;  // row tiles and K slices of a CTA, CTAs of a cluster
  int parts;            // 64-wide parts of K
  int cta_parts, warp_parts;  // ... of a CTA's and of a warp's slice (multiples of 4)
  int blocks;           // of 16 wr rows
  int t0;               // this launch's first token
  int off_sum, off_xs, off_red;  // shared memory: x, then sums, scales, partial results
  int vec;              // a row's scales can be read four at a time
};

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
// codes p and p + 4 of a word of eight as a pair of operands
template <bool BF>
__device__ __forceinline__ uint32_t codes_of(uint32_t w, int p) {
  const uint32_t c = (w >> (4 * p)) & 0x000f000fu;
  return BF ? c | 0x43004300u : c;
}
__device__ __forceinline__ float value16(uint16_t b, bool bf) {
  return bf ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}

// eight values of x, as 16 bits (bf16, or fp16), from element i of a row on
__device__ __forceinline__ void load_x8(const Linear4Params& p, const void* row, int i,
                                        uint16_t (&v)[8]) {
  if (p.x_dtype == STEP_BF16 || p.x_dtype == STEP_F16) {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + i);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (uint16_t)(u[e / 2] >> (16 * (e & 1)));
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(row) + i);
    const uint32_t u[2] = {a.x, a.y};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint8_t b = (uint8_t)(u[e / 4] >> (8 * (e & 3)));
      v[e] = p.x_dtype == STEP_E4M3 ? __nv_cvt_fp8_to_halfraw(b, __NV_E4M3).x
                                    : __half_as_ushort(__int2half_rn((int8_t)b));
    }
  }
}

// NT blocks of 8 tokens.  XS: an 8-bit x with scales below a token (else p.xs, if any,
// holds one a token).  ALONE: a warp's sums are whole (WK = C = 1).
template <int NT, bool BF, bool XS, bool ALONE>
__global__ void __launch_bounds__(32 * kWarps, NT <= 4 ? 2 : 1)
    linear4_kernel(const __grid_constant__ Plan4 q) {
  constexpr int TB = 8 * NT;
  const Linear4Params& p = q.a;
  extern __shared__ __align__(16) uint8_t smem[];
  uint16_t* sx = reinterpret_cast<uint16_t*>(smem);           // [part][half][token][j][8]
  float* ssum = reinterpret_cast<float*>(smem + q.off_sum);   // [part][token]: sums of x
  float* sxs = reinterpret_cast<float*>(smem + q.off_xs);     // [part][token]: scales of x
  float* red = reinterpret_cast<float*>(smem + q.off_red);    // partial results
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, j = lane & 3;
  const int rank = blockIdx.x % q.cluster, first = blockIdx.x / q.cluster;
  const int stride = gridDim.x / q.cluster;  // of blocks of rows
  const int tokens = min(p.T - q.t0, TB);
  const int part0 = rank * q.cta_parts, cta_parts = max(min(q.cta_parts, q.parts - part0), 0);
  const int wk = warp % q.wk, wr = warp / q.wk;
  const int my0 = wk * q.warp_parts;                                   // within the CTA's slice
  const int mine = max(min(q.warp_parts, cta_parts - my0), 0);
  const int quads = (mine + 3) / 4;
  const int rows = 16 * q.wr;

  // ---- what is ahead: four parts of 64 codes of two rows, their scales and biases
  struct Quad {
    uint2 c[4][2];
    uint2 s[2], b[2];
  };
  const long long code_pitch = p.K / 2;
  const int sgroups = p.K / p.group, per = p.group / 64;  // scales of a row; parts of a scale
  auto fetch = [&](int block, int quad, Quad& f) {
    const int o0 = block * rows + wr * 16 + g;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int o = min(o0 + 8 * h, p.O - 1);
      const int at = part0 + my0 + quad * 4;
      const uint8_t* src = p.codes + o * code_pitch + (long long)at * 32 + j * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (quad * 4 + i < mine) f.c[i][h] = __ldg(reinterpret_cast<const uint2*>(src + i * 32));
      const long long so = (long long)o * sgroups;
      if (q.vec) {
        f.s[h] = __ldg(reinterpret_cast<const uint2*>(p.scale + so + at));
        f.b[h] = __ldg(reinterpret_cast<const uint2*>(p.bias + so + at));
      } else {
        uint32_t s[4] = {0, 0, 0, 0}, b[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (quad * 4 + i < mine) {
            const int at_s = (at + i) / per;
            s[i] = __ldg(p.scale + so + at_s);
            b[i] = __ldg(p.bias + so + at_s);
          }
        f.s[h] = make_uint2(s[0] | s[1] << 16, s[2] | s[3] << 16);
        f.b[h] = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
      }
    }
  };
  int fb = first, fq = 0;  // the next quad to fetch
  Quad ring[2];
  auto next = [&](Quad& f) {
    if (fb >= q.blocks || quads == 0) return;
    fetch(fb, fq, f);
    if (++fq == quads) {
      fq = 0;
      fb += stride;
    }
  };
  next(ring[0]);
  next(ring[1]);

  // ---- the tokens' values of this CTA's slice, in the products' order
  for (int i = threadIdx.x; i < cta_parts * 8 * TB; i += 32 * kWarps) {
    // eight values: e8-th of a part's eight (j = e8 / 2, half = e8 & 1)
    const int e8 = i & 7, t = (i >> 3) % TB, part = (i >> 3) / TB;
    uint16_t v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (t < tokens) {
      const long long o = (long long)(q.t0 + t) * p.x_ts;
      const int es = p.x_dtype <= STEP_F16 ? 2 : 1;
      load_x8(p, static_cast<const uint8_t*>(p.x) + o * es, (part0 + part) * 64 + e8 * 8, v);
    }
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += value16(v[e], BF);
    // (the eight threads of a part of a token are lanes of one warp)
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
    uint4 u;
    u.x = v[0] | (uint32_t)v[4] << 16;
    u.y = v[1] | (uint32_t)v[5] << 16;
    u.z = v[2] | (uint32_t)v[6] << 16;
    u.w = v[3] | (uint32_t)v[7] << 16;
    *reinterpret_cast<uint4*>(sx + ((((part * 2 + (e8 & 1)) * TB + t) * 4 + (e8 >> 1)) << 3)) = u;
    if (e8 == 0) {
      ssum[part * TB + t] = sum;
      if (XS)
        sxs[part * TB + t] =
            t < tokens ? p.xs[(long long)(q.t0 + t) * (p.K / p.xg) + (part0 + part) * 64 / p.xg] : 0.f;
    }
  }
  __syncthreads();

  const bool bf_scale = p.bf_scale;
  float tot[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) tot[n][e] = 0.f;

  auto compute = [&](const Quad& f, int quad) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int part = my0 + quad * 4 + i;
      if (quad * 4 + i >= mine) break;
      float acc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t w0 = half ? f.c[i][0].y : f.c[i][0].x, w1 = half ? f.c[i][1].y : f.c[i][1].x;
        uint32_t a[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          a[k][0] = codes_of<BF>(w0, 2 * k);
          a[k][1] = codes_of<BF>(w1, 2 * k);
          a[k][2] = codes_of<BF>(w0, 2 * k + 1);
          a[k][3] = codes_of<BF>(w1, 2 * k + 1);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 b = *reinterpret_cast<const uint4*>(
              sx + ((((part * 2 + half) * TB + n * 8 + g) * 4 + j) << 3));
          mma16816<BF>(acc[n], a[0], b.x, b.y);
          mma16816<BF>(acc[n], a[1], b.z, b.w);
        }
      }
      float s[2], b[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t sw = i < 2 ? f.s[h].x : f.s[h].y, bw = i < 2 ? f.b[h].x : f.b[h].y;
        s[h] = value16((uint16_t)(sw >> (16 * (i & 1))), bf_scale);
        b[h] = value16((uint16_t)(bw >> (16 * (i & 1))), bf_scale);
        if (BF) b[h] = fmaf(-128.f, s[h], b[h]);
        else s[h] *= 16777216.f;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 x = *reinterpret_cast<const float2*>(ssum + part * TB + n * 8 + 2 * j);
        if constexpr (XS) {
          const float2 z = *reinterpret_cast<const float2*>(sxs + part * TB + n * 8 + 2 * j);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            tot[n][e] = fmaf(e & 1 ? z.y : z.x, fmaf(s[e >> 1], acc[n][e], b[e >> 1] * (e & 1 ? x.y : x.x)),
                             tot[n][e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            tot[n][e] = fmaf(s[e >> 1], acc[n][e], fmaf(b[e >> 1], e & 1 ? x.y : x.x, tot[n][e]));
        }
      }
    }
  };

  // y of a block: `parts` partial results at `src` (a warp's own, a CTA's, the cluster's)
  auto put = [&](int t, int o, float v) {
    if (!XS && p.xs) v *= __ldg(p.xs + q.t0 + t);
    const long long at = (q.t0 + t) * p.y_ts + o;
    if (p.y_dtype == STEP_BF16) static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
    else if (p.y_dtype == STEP_F16) static_cast<__half*>(p.y)[at] = __float2half_rn(v);
    else static_cast<float*>(p.y)[at] = v;
  };

  int buf = 0;
  for (int block = first; block < q.blocks; block += stride) {
    for (int quad = 0; quad < quads; quad += 2) {
      compute(ring[0], quad);
      next(ring[0]);
      if (quad + 1 < quads) {
        compute(ring[1], quad + 1);
        next(ring[1]);
      } else {  // an odd number of quads: the other one comes first in the next block
        const Quad x = ring[0];
        ring[0] = ring[1];
        ring[1] = x;
      }
    }
    // partial results of a warp: [token][row], rows of 16 and padding of 4 floats
    constexpr int PITCH = 20;
    float* out = red + ((ALONE ? 0 : buf) * kWarps + warp) * TB * PITCH;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        out[(n * 8 + 2 * j + (e & 1)) * PITCH + g + 8 * (e >> 1)] = tot[n][e];
        tot[n][e] = 0.f;
      }
    if constexpr (ALONE) {
      __syncwarp();
      const int o = block * rows + wr * 16 + (lane & 15);
      if (o < p.O)
        for (int t = lane >> 4; t < tokens; t += 2) put(t, o, out[t * PITCH + (lane & 15)]);
      __syncwarp();
    } else {
      if (q.cluster > 1) {
        asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
      } else {
        __syncthreads();
      }
      // this CTA's share: every cluster-th group of 16 rows x tokens
      const uint32_t at0 = smem_u32(red) + (uint32_t)(buf * kWarps * TB * PITCH) * 4;
      const int items = q.wr * tokens * 16;
      for (int i = rank * 32 * kWarps + threadIdx.x; i < items; i += q.cluster * 32 * kWarps) {
        const int r = i & 15, tile = (i >> 4) % q.wr, t = (i >> 4) / q.wr;
        const int o = block * rows + tile * 16 + r;
        float v = 0.f;
        for (int c = 0; c < q.cluster; ++c) {
          const uint32_t base = q.cluster > 1 ? mapa_shared(at0, c) : at0;
          for (int k = 0; k < q.wk; ++k) {
            float x;
            const uint32_t a = base + (uint32_t)(((tile * q.wk + k) * TB + t) * PITCH + r) * 4;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
            v += x;
          }
        }
        if (o < p.O) put(t, o, v);
      }
      buf ^= 1;  // (the next block's results go to the other buffer, the one after waits above)
    }
  }
  // no CTA of a cluster leaves while another may read its shared memory
  if (!ALONE && q.cluster > 1)
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

template <int NT, bool BF, bool XS, bool ALONE>
cudaError_t launch_t(const Plan4& q, int grid, int smem, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem((const void*)linear4_kernel<NT, BF, XS, ALONE>, 232448 - 1024, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3(32 * kWarps);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = q.cluster;
  a[0].val.clusterDim.y = 1;
  a[0].val.clusterDim.z = 1;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, linear4_kernel<NT, BF, XS, ALONE>, q);
}
template <int NT>
cudaError_t launch_nt(const Plan4& q, int grid, int smem, cudaStream_t st) {
  const bool alone = q.wk == 1 && q.cluster == 1, bf = q.a.x_dtype == STEP_BF16;
  const bool xs = q.a.xs && q.a.xg < q.a.K;
  if (bf) return alone ? launch_t<NT, true, false, true>(q, grid, smem, st) : launch_t<NT, true, false, false>(q, grid, smem, st);
  if (xs) return alone ? launch_t<NT, false, true, true>(q, grid, smem, st) : launch_t<NT, false, true, false>(q, grid, smem, st);
  return alone ? launch_t<NT, false, false, true>(q, grid, smem, st) : launch_t<NT, false, false, false>(q, grid, smem, st);
}

int round4(int x) { return (x + 3) / 4 * 4; }

}  // namespace

cudaError_t launch_linear4(const Linear4Params& p, cudaStream_t st) {
  const int sms = device_sms();
  Plan4 q{};
  q.a = p;
  q.parts = p.K / 64;
  // tokens of a launch: as many as shared memory holds beside an eighth of K
  constexpr int kRoom = 200 * 1024;
  int nt = 8;
  while (nt > 1 && 8 * (nt / 2) >= p.T) nt /= 2;
  if (nt == 8 && p.T <= 48) nt = 6;
  auto per_part = [](int nt) { return 8 * nt * (128 + 8); };
  auto red_bytes = [](int nt, bool alone) { return (alone ? 1 : 2) * kWarps * 8 * nt * 20 * 4; };
  while (nt > 1 && (long long)round4((q.parts + 7) / 8) * per_part(nt) + red_bytes(nt, false) > kRoom)
    nt = nt == 6 ? 4 : nt / 2;
  const int tiles = (p.O + 15) / 16;
  // CTAs of a cluster: while the slice of K does not fit, or there are fewer row tiles
  // than two warps of every SM would take and a warp has more than four parts
  q.cluster = 1;
  auto slice = [&](int c) { return round4((q.parts + c - 1) / c); };
  while (q.cluster < 8 && (long long)slice(q.cluster) * per_part(nt) + red_bytes(nt, false) > kRoom) q.cluster *= 2;
  // slices of K in a CTA: until there are four warps for every SM's scheduler
  q.wk = 1;
  while (q.wk < 8 && (long long)tiles * q.wk * q.cluster < 16ll * sms && slice(q.cluster) / q.wk > 4) q.wk *= 2;
  q.wr = kWarps / q.wk;
  q.cta_parts = slice(q.cluster);
  q.warp_parts = round4((q.cta_parts + q.wk - 1) / q.wk);
  q.blocks = (tiles + q.wr - 1) / q.wr;
  q.vec = p.group == 64 && q.parts % 4 == 0;
  q.off_sum = q.cta_parts * 8 * nt * 128;
  q.off_xs = q.off_sum + q.cta_parts * 8 * nt * 4;
  q.off_red = q.off_xs + q.cta_parts * 8 * nt * 4;
  const int smem = q.off_red + red_bytes(nt, q.wk == 1 && q.cluster == 1);
  const int per_sm = std::max(1, std::min(nt <= 4 ? 2 : 1, 227 * 1024 / (smem + 1024)));
  const int most = std::max(1, sms * per_sm / q.cluster);
  // (blocks evenly: no more CTAs than the rounds need)
  const int rounds = (q.blocks + most - 1) / most;
  const int grid = (q.blocks + rounds - 1) / rounds * q.cluster;
  for (q.t0 = 0; q.t0 < p.T; q.t0 += 8 * nt) {
    cudaError_t e = cudaSuccess;
    switch (nt) {
      case 1: e = launch_nt<1>(q, grid, smem, st); break;
      case 2: e = launch_nt<2>(q, grid, smem, st); break;
      case 4: e = launch_nt<4>(q, grid, smem, st); break;
      case 6: e = launch_nt<6>(q, grid, smem, st); break;
      default: e = launch_nt<8>(q, grid, smem, st); break;
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
