// The residual's addition with the RMS norm (include/step.h).
//
//   s = x + r,  n = s rsqrt(mean(s^2) + eps) w;  sum <- s, y <- n (or n in 8 bits
//   with a scale for each group of features).
//
// Bound: HBM (x, r, s and y once, some 5 operations an element); a call of a few rows
// is one launch's latency.  A row is read once and stays in registers, W warps to a
// row: one where there are many short rows (no barrier, a row's loads all in flight at
// once), eight or 32 where rows are few or long.  A group's largest magnitude is kept
// as the bits of a non-negative number, whose order as integers puts NaN above
// infinity, so that neither is lost in a maximum.
#include <algorithm>

#include "paged_internal.h"
#include "step_internal.h"

namespace moe {
namespace {

template <typename T>
struct Io;
template <>
struct Io<__nv_bfloat16> {
  static __device__ __forceinline__ float get(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
  static __device__ __forceinline__ uint16_t put(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
};
template <>
struct Io<__half> {
  static __device__ __forceinline__ float get(uint16_t b) { return __half2float(__ushort_as_half(b)); }
  static __device__ __forceinline__ uint16_t put(float v) { return __half_as_ushort(__float2half_rn(v)); }
};

// VEC values of a row from feature i on, as fp32
template <typename T, int VEC>
__device__ __forceinline__ void load_row(const void* base, long long i, float (&v)[VEC]) {
  if constexpr (sizeof(T) == 4) {
    const float* p = static_cast<const float*>(base) + i;
    if constexpr (VEC == 8) {
      const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      v[0] = *p;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + i;
    if constexpr (VEC == 8) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = Io<T>::get((uint16_t)(u[e / 2] >> (16 * (e & 1))));
    } else {
      v[0] = Io<T>::get(*p);
    }
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_row(void* base, long long i, const float (&v)[VEC]) {
  if constexpr (sizeof(T) == 4) {
    float* p = static_cast<float*>(base) + i;
    if constexpr (VEC == 8) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *p = v[0];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(base) + i;
    if constexpr (VEC == 8) {
      uint32_t u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = Io<T>::put(v[2 * e]) | (uint32_t)Io<T>::put(v[2 * e + 1]) << 16;
      *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
      *p = Io<T>::put(v[0]);
    }
  }
}
// n / scale in 8 bits (0 where the scale is); NaN stays NaN in e4m3 and is 0 in int8,
// whose scale says it
__device__ __forceinline__ uint8_t put8(float n, float scale, bool e4m3) {
  const float q = scale == 0.f ? 0.f : n / scale;
  if (e4m3) return __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
  return (uint8_t)(int8_t)min(max(__float2int_rn(q), -127), 127);
}

// The sum (or the largest value) over the W warps of a row, in every thread.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* sh) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if constexpr (W > 1) {
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += sh[w];
  }
  return v;
}

constexpr int kRowsCta = 4;  // rows of a CTA whose rows are a warp's each

// CH chunks of VEC features a thread; a CTA has one row of W warps, or kRowsCta of one.
// Q: y is 8-bit (row_max: the largest magnitudes of a row's groups, for W > 1 and for
// groups that a warp's lanes do not divide evenly).
template <typename T, int VEC, int W, int CH, bool Q>
__global__ void __launch_bounds__(W == 1 ? 32 * kRowsCta : 32 * W)
    norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int ROWS = W == 1 ? kRowsCta : 1, THREADS = 32 * W;
  __shared__ float sh_sum[W];
  extern __shared__ uint32_t row_max[];  // [ROWS][groups]
  const int tid = W == 1 ? threadIdx.x & 31 : threadIdx.x, slot = W == 1 ? threadIdx.x >> 5 : 0;
  const long long row = (long long)blockIdx.x * ROWS + slot;
  if (W == 1 && row >= (long long)p.T * p.H) return;
  const int t = (int)(row / p.H), h = (int)(row - (long long)t * p.H);
  const long long xo = t * p.x_ts + h * p.x_hs, yo = t * p.y_ts + h * p.y_hs;
  const int d = p.d;
  float v[CH][VEC];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * THREADS + tid) * VEC;
    if (i < d) {
      load_row<T, VEC>(p.x, xo + i, v[c]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[c][e] = 0.f;
    }
  }
  if (p.r) {
    const long long ro = t * p.r_ts + h * p.r_hs, so = t * p.s_ts + h * p.s_hs;
    float r[CH][VEC];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * THREADS + tid) * VEC;
      if (i < d) load_row<T, VEC>(p.r, ro + i, r[c]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * THREADS + tid) * VEC;
      if (i >= d) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[c][e] += r[c][e];
      store_row<T, VEC>(p.sum, so + i, v[c]);
    }
  }
  float sq = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < VEC; ++e) sq = fmaf(v[c][e], v[c][e], sq);
  // (the sum's barrier also puts every read of the row ahead of the first write of y,
  // which may be x)
  sq = row_sum<W>(sq, sh_sum);
  const float inv = rsqrtf(sq / (float)d + p.eps);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * THREADS + tid) * VEC;
    if (i >= d) continue;
    float w[VEC];
    if (!p.w) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] = 1.f;
    } else if (p.w_dtype == STEP_F32) {
      load_row<float, VEC>(p.w, i, w);
    } else {
      load_row<T, VEC>(p.w, i, w);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[c][e] = v[c][e] * inv * (w[e] + p.offset);
  }
  if constexpr (!Q) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * THREADS + tid) * VEC;
      if (i >= d) continue;
      if (p.y_dtype == STEP_BF16) store_row<__nv_bfloat16, VEC>(p.y, yo + i, v[c]);
      else if (p.y_dtype == STEP_F16) store_row<__half, VEC>(p.y, yo + i, v[c]);
      else store_row<float, VEC>(p.y, yo + i, v[c]);
    }
  } else {
    const int groups = d / p.group;
    uint32_t* mx = row_max + slot * groups;
    for (int g = tid; g < groups; g += THREADS) mx[g] = 0;
    if (W == 1) __syncwarp(); else __syncthreads();
    // Lanes of a group meet in shuffles first where a power of two of them holds it.
    const int lanes = p.group / VEC;
    const bool even = p.group % VEC == 0 && ((lanes & (lanes - 1)) == 0 || lanes % 32 == 0);
    const int width = min(lanes & -lanes, 32);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * THREADS + tid) * VEC;
      if (even) {
        uint32_t m = 0;
        if (i < d) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) m = max(m, __float_as_uint(v[c][e]) & 0x7fffffffu);
        }
        for (int s = width / 2; s; s >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
        if (i < d && (tid & (width - 1)) == 0) atomicMax(mx + i / p.group, m);
      } else if (i < d) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          atomicMax(mx + (i + e) / p.group, __float_as_uint(v[c][e]) & 0x7fffffffu);
      }
    }
    if (W == 1) __syncwarp(); else __syncthreads();
    const bool e4m3 = p.y_dtype == STEP_E4M3;
    const float top = e4m3 ? 448.f : 127.f;
    for (int g = tid; g < groups; g += THREADS)
      p.scales[row * groups + g] = __uint_as_float(mx[g]) / top;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * THREADS + tid) * VEC;
      if (i >= d) continue;
      uint8_t* dst = static_cast<uint8_t*>(p.y) + yo + i;
      if constexpr (VEC == 8) {
        uint32_t q[2] = {0, 0};
        if (p.group % VEC == 0) {
          const float s = __uint_as_float(mx[i / p.group]) / top;
#pragma unroll
          for (int e = 0; e < VEC; ++e) q[e / 4] |= (uint32_t)put8(v[c][e], s, e4m3) << (8 * (e & 3));
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            q[e / 4] |= (uint32_t)put8(v[c][e], __uint_as_float(mx[(i + e) / p.group]) / top, e4m3)
                        << (8 * (e & 3));
        }
        *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
      } else {
        *dst = put8(v[c][0], __uint_as_float(mx[i / p.group]) / top, e4m3);
      }
    }
  }
}

template <typename T, int VEC, int W, int CH>
cudaError_t norm_launch(const NormParams& p, cudaStream_t st) {
  constexpr int ROWS = W == 1 ? kRowsCta : 1;
  const long long rows = (long long)p.T * p.H;
  const dim3 grid((unsigned)((rows + ROWS - 1) / ROWS)), block(W == 1 ? 32 * ROWS : 32 * W);
  if (p.y_dtype != STEP_E4M3 && p.y_dtype != STEP_I8)
    return launch_kernel(norm_kernel<T, VEC, W, CH, false>, grid, block, 0, st, p);
  const int smem = ROWS * (p.d / p.group) * 4;
  static std::atomic<uint64_t> allowed{0};
  if (smem > 40000) {
    const cudaError_t e = allow_smem((const void*)norm_kernel<T, VEC, W, CH, true>, 4 * kNormMaxD + 1024, allowed);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(norm_kernel<T, VEC, W, CH, true>, grid, block, smem, st, p);
}

bool aligned_to(const void* p, long long a, long long b, int es, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) % bytes) == 0 && a * es % bytes == 0 && b * es % bytes == 0;
}

// A warp to a row while a warp of every SM has one: 8192 rows of 2048 and more; eight
// warps shorten the latency of fewer.
template <typename T>
cudaError_t norm_by_shape(const NormParams& p, cudaStream_t st) {
  const int es = sizeof(T), ys = p.y_dtype == STEP_F32 ? 4 : p.y_dtype <= STEP_F16 ? 2 : 1;
  const bool vec = p.d % 8 == 0 && aligned_to(p.x, p.x_ts, p.x_hs, es, 16) &&
                   (!p.r || (aligned_to(p.r, p.r_ts, p.r_hs, es, 16) && aligned_to(p.sum, p.s_ts, p.s_hs, es, 16))) &&
                   aligned_to(p.w, 0, 0, 1, 16) &&
                   aligned_to(p.y, p.y_ts, p.y_hs, ys, ys == 1 ? 8 : 16);
  const long long rows = (long long)p.T * p.H;
  const bool many = rows >= 4ll * device_sms();
  if (vec) {
    if (p.d <= 256) return norm_launch<T, 8, 1, 1>(p, st);
    if (p.d <= 1024 && many) return norm_launch<T, 8, 1, 4>(p, st);
    if (p.d <= 2048) return many ? norm_launch<T, 8, 1, 8>(p, st) : norm_launch<T, 8, 8, 1>(p, st);
    if (p.d <= 8192) return norm_launch<T, 8, 8, 4>(p, st);
    return norm_launch<T, 8, 32, 4>(p, st);
  }
  if (p.d <= 256) return norm_launch<T, 1, 1, 8>(p, st);
  if (p.d <= 2048) return norm_launch<T, 1, 8, 8>(p, st);
  return norm_launch<T, 1, 32, 32>(p, st);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t st) {
  if (p.dtype == STEP_BF16) return norm_by_shape<__nv_bfloat16>(p, st);
  if (p.dtype == STEP_F16) return norm_by_shape<__half>(p, st);
  return norm_by_shape<float>(p, st);
}

}  // namespace moe
