// Products of a few tokens with 4-bit weights in the checkpoint's layout
// (include/step.h).
//
//   y[t][o] = sum over groups of (s sum c x + b sum x)
// so the products of a group run on the codes themselves, which are exact in 16 bits,
// and scale and bias enter once a group in fp32:
//   bf16:  a code behind the leading bit of 16 is 16 + c, and the group's sum is
//          s acc + (b - 16 s) X with X = sum x
//   fp16 (8-bit x too, which fp16 holds exactly):  a code's bits alone are the subnormal
//          c 2^-24, and the group's sum is (2^24 s) acc + b X
// An 8-bit x has its own scale applied after a 64-wide part (or at the end, where a
// token has one).
//
// Floor: HBM (half a byte a weight plus four a group).  For up to 8 tokens over a vocabulary no
// unit is full: DRAM 52 %, the ALU 48 % and the issue slots 58 % of the cycles in which an SM
// works, with 16 warps of 116 registers an SM (22 % of what it holds) to hide one another's
// waits.  From 16 tokens on it is the instructions that turn codes into operands, some 95 a part of
// 16 x 64 weights, done anew for every 16 tokens (8 where K is above 16384, whose tokens no eighth
// of K leaves room for).  A warp has 16 rows of weights as the
// wide side of mma.sync (m16n8k16) and 8 or 16 tokens as the narrow one; more tokens are
// further CTAs' (up to 64 of a warp were slower at every size: registers and reads of the
// tokens).  Lane (g, j) of a warp takes rows g and g + 8 and of each part of 64 weights the
// codes 16 j .. 16 j + 15, 8 bytes a row, which shifts turn into operands in the order
// 0 4 1 5 2 6 3 7; the tokens are laid out in shared memory in that order once.  A warp's rows
// come through a ring of its own by 16-byte copies, four parts a stage (2.3 KB), two stages
// ahead and across blocks of rows, so that a CTA that walks many never drains.  (The same
// loads into registers took 123 instructions a part, and 70 us for 130001 x 2048 weights
// and 8 tokens.)
//
// Split: a CTA, one an SM, holds WR row tiles x WK slices of K (WR WK = 16 warps), and a
// cluster of C CTAs splits K again where the tokens of all of K do not fit shared memory;
// partial sums meet in shared memory, in a fixed order.
// Measured (a graph replay's time, weights not in L2, of which some 5 us are the method's):
// 5120 x 2048, one token 11.4 us, 8 13.4, 64 23.7; 2047 x 4096, 37 tokens of e4m3 21.6;
// 130001 x 2048 (150 MB), one token 42, 8 42 (4.1 TB/s), 16 56, 32 87, 64 157, 256 605; a product
// of 16-bit weights, 131072 of them, by the library 97, 97, 100, 100, 110 and 118.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "paged_internal.h"
#include "ptx.cuh"
#include "step_internal.h"

namespace moe {
namespace {

constexpr int kWarps = 16;
constexpr int kStages = 3;
constexpr int kPitch = 160;                   // bytes of a row of a stage: no bank conflicts
constexpr int kStage = 16 * kPitch + 16 * 16;  // codes of 16 rows x 4 parts, scales and biases

struct Plan4 {
  Linear4Params a;
  int wr, wk, cluster;  // row tiles and K slices of a CTA, CTAs of a cluster
  int parts;            // 64-wide parts of K
  int cta_parts, warp_parts;  // ... of a CTA's and of a warp's slice (multiples of 4)
  int blocks;           // of 16 wr rows
  int off_sum, off_xs, off_ring, off_red;  // shared memory: x, its sums and scales, the rest
  int vec;              // a row's scales can be read four at a time
};

// c = a b + c, or a b alone.  (Not volatile: the products of a stage's parts, which do not
// depend on one another, may pass each other.)
template <bool BF, bool ADD>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  const float z[4] = {ADD ? c[0] : 0.f, ADD ? c[1] : 0.f, ADD ? c[2] : 0.f, ADD ? c[3] : 0.f};
  if constexpr (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z[0]), "f"(z[1]), "f"(z[2]),
          "f"(z[3]));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z[0]), "f"(z[1]), "f"(z[2]),
          "f"(z[3]));
}
// codes p and p + 4 of a word of eight as a pair of operands
template <bool BF>
struct Codes {
  uint32_t mask, lead;  // (in registers: as literals they take an AND and an OR, or moves)
  __device__ Codes() {
    asm volatile("mov.b32 %0, 0x00780078;" : "=r"(mask));
    asm volatile("mov.b32 %0, 0x41804180;" : "=r"(lead));
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t w, int p) const {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
        : "=r"(r) : "r"(p == 0 ? w << 3 : w >> (4 * p - 3)), "r"(mask), "r"(lead));
    return r;
  }
};
template <>
struct Codes<false> {
  __device__ __forceinline__ uint32_t operator()(uint32_t w, int p) const {
    return (w >> (4 * p)) & 0x000f000fu;
  }
};
__device__ __forceinline__ float value16(uint16_t b, bool bf) {
  return bf ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}

// eight values of x from element i of a row on, as they lie in memory, and as 16 bits
// (bf16, or fp16)
__device__ __forceinline__ uint4 raw_x8(const Linear4Params& p, long long i) {
  if (p.x_dtype <= STEP_F16)
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + i));
  const uint2 a = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.x) + i));
  return make_uint4(a.x, a.y, 0, 0);
}
__device__ __forceinline__ void unpack_x8(int dtype, uint4 a, uint16_t (&v)[8]) {
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
  if (dtype <= STEP_F16) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (uint16_t)(u[e / 2] >> (16 * (e & 1)));
  } else {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const uint16_t b = (uint16_t)(u[e / 4] >> (8 * (e & 3)));
      if (dtype == STEP_E4M3) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(b, __NV_E4M3);
        v[e] = h.x, v[e + 1] = h.y;
      } else {
        v[e] = __half_as_ushort(__int2half_rn((int8_t)b));
        v[e + 1] = __half_as_ushort(__int2half_rn((int8_t)(b >> 8)));
      }
    }
  }
}

// NT blocks of 8 tokens.  XS: an 8-bit x with scales below a token (else p.xs, if any,
// holds one a token).  ALONE: a warp's sums are whole (WK = C = 1).
template <int NT, bool BF, bool XS, bool ALONE>
__global__ void __launch_bounds__(32 * kWarps, 1)
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
  const int t0 = blockIdx.y * TB, tokens = min(p.T - t0, TB);
  const int part0 = rank * q.cta_parts, cta_parts = max(min(q.cta_parts, q.parts - part0), 0);
  const int wk = warp % q.wk, wr = warp / q.wk;
  const int my0 = wk * q.warp_parts;                                   // within the CTA's slice
  const int mine = max(min(q.warp_parts, cta_parts - my0), 0);
  const int quads = (mine + 3) / 4;
  const int rows = 16 * q.wr;

  // ---- the ring: stage i of a warp's sequence (blocks of rows, of each its quads of parts)
  uint8_t* const ring = smem + q.off_ring + warp * kStages * kStage;
  const uint32_t ring_at = smem_u32(ring);
  const long long code_pitch = p.K / 2;
  const int sgroups = p.K / p.group, per = p.group / 64;  // scales of a row; parts of a scale
  int fb = first, fq = 0;  // the next block and quad to copy
  // A lane copies 16 bytes of rows lane / 8, + 4, + 8 and + 12 of a stage, and the four
  // scales or biases of row lane / 2: from these addresses on, which move with the quads.
  const uint8_t* code_src = nullptr;
  const uint16_t* scale_src = nullptr;
  const int code_dst = (lane >> 3) * kPitch + (lane & 7) * 16;
  const int part_first = part0 + my0;
  int row_left = 0;  // rows of the block behind this lane's first
  // the first row of this warp's tile of a block
  auto row_of = [&](int block) {
    return ALONE ? ((block - first) * kWarps + wr * stride + first) * 16 : block * rows + wr * 16;
  };
  auto enter = [&]() {
    const int o0 = row_of(fb);
    row_left = p.O - o0 - (lane >> 3);
    code_src = p.codes + (o0 + (lane >> 3)) * code_pitch + (long long)part_first * 32 + (lane & 7) * 16;
    scale_src = (lane & 1 ? p.bias : p.scale) + (long long)min(o0 + (lane >> 1), p.O - 1) * sgroups;
    if (q.vec) scale_src += part_first;
  };
  enter();
  uint2 pending = make_uint2(0, 0);  // scales whose rows are not 8-byte aligned come by way of
  int pending_at = -1;               // registers, a stage later
  auto fetch = [&](int slot) {
    if (!q.vec && pending_at >= 0) {
      *reinterpret_cast<uint2*>(ring + pending_at + lane * 8) = pending;
      pending_at = -1;
    }
    if (fb < q.blocks && quads > 0) {
      const uint32_t dst = ring_at + slot * kStage;
      const int left = (mine - fq * 4) * 2;  // 16-byte pieces of a row
      if (left >= 8 && row_left > 12) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          cp_async16(dst + code_dst + i * 4 * kPitch, code_src + i * 4 * code_pitch, 16u);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool is = row_left > 4 * i && (lane & 7) < left;
          cp_async16(dst + code_dst + i * 4 * kPitch, is ? code_src + i * 4 * code_pitch : p.codes,
                     is ? 16u : 0u);
        }
      }
      code_src += 128;
      if (q.vec) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst + 16 * kPitch + lane * 8),
                     "l"(scale_src) : "memory");
        scale_src += 4;
      } else {
        uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (2 * i < left) v[i] = __ldg(scale_src + (part_first + fq * 4 + i) / per);
        pending = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
        pending_at = slot * kStage + 16 * kPitch;
      }
      if (++fq == quads) {
        fq = 0;
        fb += stride;
        enter();
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);

  // ---- the tokens' values of this CTA's slice, in the products' order
  // (eight loads of a thread in flight; eight values a step: the e8-th eight of a part of
  // token t, which lane j = e8 / 2 of the products takes)
  constexpr int AHEAD = 8;
  const int items = cta_parts * 8 * TB;
  for (int base = threadIdx.x; base < items; base += AHEAD * 32 * kWarps) {
    uint4 raw[AHEAD];
    float z[AHEAD];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int i = base + a * 32 * kWarps;
      const int e8 = i & 7, t = (i >> 3) % TB, part = part0 + (i >> 3) / TB;
      raw[a] = make_uint4(0, 0, 0, 0);
      z[a] = 0.f;
      if (i < items && t < tokens) {
        raw[a] = raw_x8(p, (t0 + t) * p.x_ts + part * 64 + e8 * 8);
        if (XS && e8 == 0) z[a] = __ldg(p.xs + (long long)(t0 + t) * (p.K / p.xg) + part * 64 / p.xg);
      }
    }
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int i = base + a * 32 * kWarps;
      if (i >= items) break;  // (the same for a warp: items are a multiple of 64)
      const int e8 = i & 7, t = (i >> 3) % TB, part = (i >> 3) / TB;
      uint16_t v[8];
      unpack_x8(p.x_dtype, raw[a], v);
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
        if (XS) sxs[part * TB + t] = z[a];
      }
    }
  }
  __syncthreads();

  const bool bf_scale = p.bf_scale;
  float tot[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) tot[n][e] = 0.f;

  // A stage's four parts (`left` of them, FULL: all) from part `quad * 4` of the slice on.
  // This lane's operands lie at fixed distances from three addresses.
  const uint8_t* const x_lane = smem + (g * 4 + j) * 16;
  const float* const sum_lane = ssum + 2 * j;
  const float* const xs_lane = sxs + 2 * j;
  const int code_lane = g * kPitch + j * 8;
  const Codes<BF> codes;
  auto compute = [&](const uint8_t* st, int quad, int left, auto full) {
    constexpr bool FULL = decltype(full)::value;
    const int part0 = my0 + quad * 4;
    const uint8_t* const xq = x_lane + part0 * (TB * 128);
    const float* const sq = sum_lane + part0 * TB;
    [[maybe_unused]] const float* const zq = xs_lane + part0 * TB;
    float s[4][2], b[4][2];  // of rows g and g + 8
    uint32_t u[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 v = *reinterpret_cast<const uint4*>(st + 16 * kPitch + (g + 8 * h) * 16);
      u[h][0] = v.x, u[h][1] = v.y, u[h][2] = v.z, u[h][3] = v.w;
    }
    if (bf_scale) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[i][h] = __uint_as_float(i & 1 ? u[h][i / 2] & 0xffff0000u : u[h][i / 2] << 16);
          b[i][h] = __uint_as_float(i & 1 ? u[h][2 + i / 2] & 0xffff0000u : u[h][2 + i / 2] << 16);
        }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&u[h][i / 2]));
          const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&u[h][2 + i / 2]));
          s[i][h] = x.x, s[i + 1][h] = x.y, b[i][h] = y.x, b[i + 1][h] = y.y;
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (BF) b[i][h] = fmaf(-16.f, s[i][h], b[i][h]);
        else s[i][h] *= 16777216.f;
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!FULL && i >= left) break;
      const uint2 c0 = *reinterpret_cast<const uint2*>(st + code_lane + i * 32);
      const uint2 c1 = *reinterpret_cast<const uint2*>(st + code_lane + 8 * kPitch + i * 32);
      float acc[NT][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t w0 = half ? c0.y : c0.x, w1 = half ? c1.y : c1.x;
        uint32_t a[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          a[k][0] = codes(w0, 2 * k);
          a[k][1] = codes(w1, 2 * k);
          a[k][2] = codes(w0, 2 * k + 1);
          a[k][3] = codes(w1, 2 * k + 1);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 x = *reinterpret_cast<const uint4*>(xq + (i * 2 + half) * (TB * 64) + n * 512);
          if (half == 0) mma16816<BF, false>(acc[n], a[0], x.x, x.y);
          else mma16816<BF, true>(acc[n], a[0], x.x, x.y);
          mma16816<BF, true>(acc[n], a[1], x.z, x.w);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 x = *reinterpret_cast<const float2*>(sq + i * TB + n * 8);
        if constexpr (XS) {
          const float2 z = *reinterpret_cast<const float2*>(zq + i * TB + n * 8);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            tot[n][e] = fmaf(e & 1 ? z.y : z.x,
                             fmaf(s[i][e >> 1], acc[n][e], b[i][e >> 1] * (e & 1 ? x.y : x.x)), tot[n][e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            tot[n][e] = fmaf(s[i][e >> 1], acc[n][e], fmaf(b[i][e >> 1], e & 1 ? x.y : x.x, tot[n][e]));
        }
      }
    }
  };

  // y of a block: `parts` partial results at `src` (a warp's own, a CTA's, the cluster's)
  auto put = [&](int t, int o, float v) {
    if (!XS && p.xs) v *= __ldg(p.xs + t0 + t);
    const long long at = (t0 + t) * p.y_ts + o;
    if (p.y_dtype == STEP_BF16) static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
    else if (p.y_dtype == STEP_F16) static_cast<__half*>(p.y)[at] = __float2half_rn(v);
    else static_cast<float*>(p.y)[at] = v;
  };

  int slot = 0;
  for (int block = first; block < q.blocks; block += stride) {
    if (ALONE && row_of(block) >= p.O) break;  // (nor has this warp a tile in later blocks)
    for (int quad = 0; quad < quads; ++quad) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // the stage is there for all lanes, and the one before has been read
      fetch(slot == 0 ? kStages - 1 : slot - 1);
      const int left = mine - quad * 4;
      if (left >= 4) compute(ring + slot * kStage, quad, 4, std::true_type{});
      else compute(ring + slot * kStage, quad, left, std::false_type{});
      if (++slot == kStages) slot = 0;
    }
    // partial results of a warp: [token][row], rows of 16 and padding of 4 floats
    constexpr int PITCH = 20;
    float* out = red + warp * TB * PITCH;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        out[(n * 8 + 2 * j + (e & 1)) * PITCH + g + 8 * (e >> 1)] = tot[n][e];
        tot[n][e] = 0.f;
      }
    if constexpr (ALONE) {
      __syncwarp();
      const int o = row_of(block) + (lane & 15);
      if (o < p.O)
        for (int t = lane >> 4; t < tokens; t += 2) put(t, o, out[t * PITCH + (lane & 15)]);
      __syncwarp();
    } else {
      if (q.cluster > 1) {
        asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
      } else {
        __syncthreads();
      }
      // this CTA's share: the tokens rank, rank + C, ...; a thread a row
      const uint32_t at0 = smem_u32(red);
      const int r = threadIdx.x % rows, o = block * rows + r, tile = r >> 4;
      if (o < p.O) {
        for (int t = rank + threadIdx.x / rows * q.cluster; t < tokens; t += 32 * kWarps / rows * q.cluster) {
          float v = 0.f;
          const uint32_t a0 = at0 + (uint32_t)((tile * q.wk * TB + t) * PITCH + (r & 15)) * 4;
          if (q.cluster == 1) {
            float x[kWarps];
#pragma unroll
            for (int k = 0; k < kWarps; ++k)
              x[k] = k < q.wk ? __uint_as_float(ld_shared_u32(a0 + k * (TB * PITCH * 4))) : 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) v += x[k];
          } else {
            for (int k = 0; k < q.wk; ++k) {
              float x[8];
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                x[c] = 0.f;
                if (c < q.cluster)
                  asm volatile("ld.shared::cluster.f32 %0, [%1];"
                               : "=f"(x[c]) : "r"(mapa_shared(a0 + k * (TB * PITCH * 4), c)) : "memory");
              }
#pragma unroll
              for (int c = 0; c < 8; ++c) v += x[c];
            }
          }
          put(t, o, v);
        }
      }
      // before the next block's results; no CTA of a cluster leaves while another may read
      // its shared memory
      if (q.cluster > 1) {
        asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
      } else {
        __syncthreads();
      }
    }
  }
  cp_async_wait<0>();
}

template <int NT, bool BF, bool XS, bool ALONE>
cudaError_t launch_t(const Plan4& q, dim3 grid, int smem, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem((const void*)linear4_kernel<NT, BF, XS, ALONE>, 232448 - 1024, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
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
cudaError_t launch_nt(const Plan4& q, dim3 grid, int smem, cudaStream_t st) {
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
  constexpr int kRing = kWarps * kStages * kStage;
  constexpr int kRoom = 226 * 1024 - kRing;  // for the tokens and the partial results
  auto slice = [&](int c) { return round4((q.parts + c - 1) / c); };
  auto bytes = [&](int c, int nt) {
    return (long long)slice(c) * 8 * nt * (128 + 8) + kWarps * 8 * nt * 20 * 4;
  };
  // 8 or 16 tokens a CTA (8 where an eighth of K leaves no room for more)
  const int nt = p.T <= 8 || bytes(8, 2) > kRoom ? 1 : 2, groups = (p.T + 8 * nt - 1) / (8 * nt);
  const int red = kWarps * 8 * nt * 20 * 4;
  const int tiles = (p.O + 15) / 16;
  // CTAs of a cluster while their slice of the tokens does not fit; slices of K in a CTA
  // until the CTAs fill more than half of the SMs, or a warp has four parts left (GPU time:
  // 2047 x 4096, one token, 16 slices 11.4 us, 8 slices 13.4, one 25.8; 12288 x 2048 2 and
  // 96 CTAs 13.4, one 17.5, 4 15.5; 32768 x 2048 one 17.6, 2 19.6).
  q.cluster = 1;
  while (q.cluster < 8 && bytes(q.cluster, nt) > kRoom) q.cluster *= 2;
  q.wk = 1;
  while (q.wk < kWarps && slice(q.cluster) > 4 * q.wk &&
         (long long)tiles * q.wk * q.cluster * groups * 10 < 6ll * sms * kWarps)
    q.wk *= 2;
  q.wr = kWarps / q.wk;
  q.cta_parts = slice(q.cluster);
  q.warp_parts = round4((q.cta_parts + q.wk - 1) / q.wk);
  q.blocks = (tiles + q.wr - 1) / q.wr;
  q.vec = p.group == 64 && q.parts % 4 == 0;
  q.off_sum = q.cta_parts * 8 * nt * 128;
  q.off_xs = q.off_sum + q.cta_parts * 8 * nt * 4;
  q.off_ring = q.off_xs + q.cta_parts * 8 * nt * 4;
  q.off_red = q.off_ring + kRing;
  const int smem = q.off_red + red;
  const int ctas = std::min(q.blocks, std::max(1, sms / q.cluster / groups));
  // (a warp alone takes every so many row tiles, so that the last round is every SM's)
  if (q.wk == 1 && q.cluster == 1) q.blocks = (tiles + kWarps * ctas - 1) / (kWarps * ctas) * ctas;
  const dim3 grid(ctas * q.cluster, groups);
  return nt == 1 ? launch_nt<1>(q, grid, smem, st) : launch_nt<2>(q, grid, smem, st);
}

}  // namespace moe
