// The residual's addition with the RMS norm (include/step.h).
//
//   s = x + r,  n = s rsqrt(mean(s^2) + eps) w;  sum <- s, y <- n (or n in 8 bits
//   with a scale for each group of features).
//
// Bound: HBM (x, r, s and y once, some 5 operations an element); a call of a few rows
// is one launch's latency.  A row is read once and stays in registers, two vectors of
// eight a thread, W warps to a row; a CTA walks over rows with the weights in registers
// and reads its next row before it is done with one.  Measured (x + r, L2 warm): 8192 rows
// of 2048 in bf16 22.7 us (134 MB, 5.9 TB/s), to e4m3 26.8 (117 MB, 4.4 TB/s), fp32 51
// (268 MB, 5.2 TB/s); 4096 of 4096 23, to e4m3 27; 65552 heads of 256, no sum, 12.5 (67 MB, of
// which L2 holds most: 15 with L2 cold), of 128 as long, since half of a warp's lanes have no
// features; 2000 of 8191, which start anywhere and take one feature a load, 41; one row 4.2.
// A group's largest magnitude is kept as the bits of a non-negative number, whose order as
// integers puts NaN above
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
  static __device__ __forceinline__ uint32_t put2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <>
struct Io<__half> {
  static __device__ __forceinline__ float get(uint16_t b) { return __half2float(__ushort_as_half(b)); }
  static __device__ __forceinline__ uint16_t put(float v) { return __half_as_ushort(__float2half_rn(v)); }
  static __device__ __forceinline__ uint32_t put2(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

// VEC values of a row from feature i on: as they lie in memory, and as fp32
template <typename T, int VEC>
struct Raw {
  static constexpr int N = VEC == 1 ? 1 : VEC * (int)sizeof(T) / 4;
  uint32_t u[N];
  __device__ __forceinline__ void load(const void* base, long long i) {
    const T* p = static_cast<const T*>(base) + i;
    if constexpr (VEC == 1) {
      if constexpr (sizeof(T) == 4) u[0] = *reinterpret_cast<const uint32_t*>(p);
      else u[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        const uint4 a = reinterpret_cast<const uint4*>(p)[k / 4];
        u[k] = a.x, u[k + 1] = a.y, u[k + 2] = a.z, u[k + 3] = a.w;
      }
    }
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(u[e]);
    else return Io<T>::get((uint16_t)(VEC == 1 ? u[0] : u[e / 2] >> (16 * (e & 1))));
  }
};
template <typename T, int VEC>
__device__ __forceinline__ void load_row(const void* base, long long i, float (&v)[VEC]) {
  Raw<T, VEC> r;
  r.load(base, i);
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = r[e];
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
      for (int e = 0; e < 4; ++e) u[e] = Io<T>::put2(v[2 * e], v[2 * e + 1]);
      *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
      *p = Io<T>::put(v[0]);
    }
  }
}
// A group's scale: its largest magnitude (as bits) / top, rounded to nearest; below fp32's
// normal numbers upwards, so that no quotient passes the type's end and no group but one of
// zeros has a scale of 0.
__device__ __forceinline__ float scale_of(uint32_t m, float top) {
  const float v = __uint_as_float(m), scale = v / top;
  return scale < 0x1p-126f ? __fdiv_ru(v, top) : scale;
}
// Eight bits: the quotient n / scale, one division a group: a product with the scale's
// reciprocal, corrected by its remainder (Markstein), so that a quotient on a border between two
// values is on it.  (The product alone is up to 1.5 steps of fp32 off.  `pre` keeps a tiny
// scale's reciprocal and remainders in fp32's range; with an infinite scale there is no
// remainder.)  NaN stays NaN in e4m3 and is 0 in int8, whose scale says it.
struct Scaler {
  float pre, by, inv;
  __device__ explicit Scaler(float scale) {
    pre = scale < 1e-20f ? 0x1p64f : 1.f;
    by = scale * pre;
    inv = scale == 0.f ? 0.f : 1.f / by;
    if (by == INFINITY) by = 0.f;
  }
  __device__ __forceinline__ float operator()(float n) const {
    const float m = n * pre, q = m * inv;
    return fmaf(-fmaf(q, by, -m), inv, q);
  }
};
__device__ __forceinline__ uint32_t put8x2(float a, float b, bool e4m3) {
  if (e4m3) return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const int x = min(max(__float2int_rn(a), -127), 127), y = min(max(__float2int_rn(b), -127), 127);
  return (x & 0xff) | (y & 0xff) << 8;
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
__global__ void __launch_bounds__(W == 1 ? 32 * kRowsCta : 32 * W, W >= 8 && CH * VEC <= 16 ? 32 / W : 1)
    norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int ROWS = W == 1 ? kRowsCta : 1, THREADS = 32 * W;
  __shared__ float sh_sum[2][W];  // by turns
  extern __shared__ uint32_t row_max[];  // [ROWS][groups]
  const int tid = W == 1 ? threadIdx.x & 31 : threadIdx.x, slot = W == 1 ? threadIdx.x >> 5 : 0;
  const int d = p.d;
  const unsigned rows = (unsigned)p.T * (unsigned)p.H;  // below 2^31 - 4
  // The weights stay in registers over a CTA's rows where they are few.
  constexpr bool HOLD = CH * VEC <= 16, PIPE = HOLD && CH > 1;
  auto weights = [&](int i, float (&w)[VEC]) {
    if (!p.w || i >= d) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] = 1.f;
    } else if (p.w_dtype == STEP_F32) {
      load_row<float, VEC>(p.w, i, w);
    } else {
      load_row<T, VEC>(p.w, i, w);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[e] += p.offset;
  };
  float hold[HOLD ? CH : 1][VEC];
  if constexpr (HOLD) {
#pragma unroll
    for (int c = 0; c < CH; ++c) weights((c * THREADS + tid) * VEC, hold[c]);
  }
  // A row's loads are all in flight before the first is waited for; where a thread holds
  // little, the next row's before this one's sum.
  Raw<T, VEC> x[CH], r[CH];
  auto load = [&](unsigned at) {
    const int t = fast_div((int)at, p.div_h), h = (int)at - t * p.H;
    const long long xo = t * p.x_ts + h * p.x_hs, ro = t * p.r_ts + h * p.r_hs;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * THREADS + tid) * VEC;
#pragma unroll
      for (int k = 0; k < x[c].N; ++k) x[c].u[k] = 0;
      if (i < d) x[c].load(p.x, xo + i);
    }
    if (!p.r) return;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * THREADS + tid) * VEC;
#pragma unroll
      for (int k = 0; k < r[c].N; ++k) r[c].u[k] = 0;
      if (i < d) r[c].load(p.r, ro + i);
    }
  };
  unsigned at = blockIdx.x * ROWS + slot;
  if (PIPE && at < rows) load(at);
  int turn = 0;
#pragma unroll 1
  for (; at < rows; at += gridDim.x * ROWS) {
    const int row = (int)at;
    const int t = fast_div(row, p.div_h), h = row - t * p.H;
    const long long yo = t * p.y_ts + h * p.y_hs;
    if (!PIPE) load(at);
    float v[CH][VEC];
    if (p.r) {
      const long long so = t * p.s_ts + h * p.s_hs;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (c * THREADS + tid) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[c][e] = x[c][e] + r[c][e];
        if (i < d) store_row<T, VEC>(p.sum, so + i, v[c]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[c][e] = x[c][e];
    }
    if (PIPE && at + gridDim.x * ROWS < rows) load(at + gridDim.x * ROWS);
    float sq = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) sq = fmaf(v[c][e], v[c][e], sq);
    // (the sum's barrier also puts every read of the row ahead of the first write of y,
    // which may be x)
    sq = row_sum<W>(sq, sh_sum[turn]);
    turn ^= 1;
    const float inv = rsqrtf(sq * p.inv_d + p.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float w[VEC];
      if constexpr (!HOLD) weights((c * THREADS + tid) * VEC, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[c][e] = v[c][e] * inv * (HOLD ? hold[c][e] : w[e]);
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
      const bool e4m3 = p.y_dtype == STEP_E4M3;
      const float top = e4m3 ? 448.f : 127.f;
      float* const scales = p.scales + (long long)row * groups;
      auto put = [&](const float (&z)[VEC], int i) {
        uint8_t* dst = static_cast<uint8_t*>(p.y) + yo + i;
        if constexpr (VEC == 8)
          *reinterpret_cast<uint2*>(dst) =
              make_uint2(put8x2(z[0], z[1], e4m3) | put8x2(z[2], z[3], e4m3) << 16,
                         put8x2(z[4], z[5], e4m3) | put8x2(z[6], z[7], e4m3) << 16);
        else *dst = (uint8_t)put8x2(z[0], 0.f, e4m3);
      };
      // A group that a power of two of a warp's lanes hold: its maximum by shuffles alone.
      const int lanes = p.group % VEC ? 0 : p.group / VEC;
      if (lanes > 0 && lanes <= 32 && (lanes & (lanes - 1)) == 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int i = (c * THREADS + tid) * VEC;
          uint32_t m = 0;
          if (i < d) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) m = max(m, __float_as_uint(v[c][e]) & 0x7fffffffu);
          }
          for (int s = lanes / 2; s; s >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
          if (i >= d) continue;
          const float scale = scale_of(m, top);
          if ((tid & (lanes - 1)) == 0) scales[fast_div(i, p.div)] = scale;
          const Scaler s(scale);
          float z[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) z[e] = s(v[c][e]);
          put(z, i);
        }
        continue;
      }
      uint32_t* mx = row_max + slot * groups;
      for (int g = tid; g < groups; g += THREADS) mx[g] = 0;
      if (W == 1) __syncwarp(); else __syncthreads();
      const bool even = lanes > 0 && lanes % 32 == 0;  // a warp's lanes of a chunk in one group
// All of a warp's maxima by shuffles before the first lane goes its own way.  (One
      // chunk after another with a warp-wide reduction instruction in place of the shuffles,
      // compiled for 64 registers, lost groups' maxima, with a __syncwarp before it too; for as many
      // registers as it likes, or in a loop of its own like this one, the same was right.)
      uint32_t m[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        m[c] = 0;
        if ((c * THREADS + tid) * VEC < d && lanes > 0) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) m[c] = max(m[c], __float_as_uint(v[c][e]) & 0x7fffffffu);
        }
      }
      if (even) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int s = 16; s; s >>= 1) m[c] = max(m[c], __shfl_xor_sync(0xffffffffu, m[c], s));
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (c * THREADS + tid) * VEC;
        if (i >= d) continue;
        if (lanes > 0) {
          if (!even || (tid & 31) == 0) atomicMax(mx + fast_div(i, p.div), m[c]);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            atomicMax(mx + fast_div(i + e, p.div), __float_as_uint(v[c][e]) & 0x7fffffffu);
        }
      }
      if (W == 1) __syncwarp(); else __syncthreads();
      for (int g = tid; g < groups; g += THREADS) scales[g] = scale_of(mx[g], top);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (c * THREADS + tid) * VEC;
        if (i >= d) continue;
        float z[VEC];
        if (lanes > 0) {
          const Scaler s(scale_of(mx[fast_div(i, p.div)], top));
#pragma unroll
          for (int e = 0; e < VEC; ++e) z[e] = s(v[c][e]);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            z[e] = Scaler(scale_of(mx[fast_div(i + e, p.div)], top))(v[c][e]);
        }
        put(z, i);
      }
      if (W == 1) __syncwarp(); else __syncthreads();  // before the next row's maxima
    }
  }
}

template <typename T, int VEC, int W, int CH>
cudaError_t norm_launch(const NormParams& p, cudaStream_t st) {
  constexpr int ROWS = W == 1 ? kRowsCta : 1;
  const long long rows = (long long)p.T * p.H;
  const bool q = p.y_dtype == STEP_E4M3 || p.y_dtype == STEP_I8;
  const dim3 block(W == 1 ? 32 * ROWS : 32 * W);
  // as many CTAs as run at once, each with its share of the rows: it prefetches its next
  // (8192 x 2048 to e4m3, when this stood at 25 us: twice as many 26.7, a CTA a row 36)
  static std::atomic<int> fit[2]{};
  int each = fit[q].load(std::memory_order_relaxed);
  if (each == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
        &each, q ? norm_kernel<T, VEC, W, CH, true> : norm_kernel<T, VEC, W, CH, false>, (int)block.x, 0);
    if (e != cudaSuccess) return e;
    each = std::max(each, 1);
    fit[q].store(each, std::memory_order_relaxed);
  }
  const dim3 grid((unsigned)std::min((rows + ROWS - 1) / ROWS, (long long)each * device_sms()));
  if (!q)
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

// As few warps a row as hold it in two vectors a thread (8192 x 2048 to e4m3, four warps
// 27 us, two with four vectors 33, eight with one 34; 4096 x 4096 eight warps 24, four 27,
// sixteen with one vector 27; 65536 x 512 one warp 46, two 47, four 56).  Where SMs have
// few rows a thread has one vector, eight warps up to 2048 features (16 x 2048 4.3 us, 6.3
// with four).  The launch bounds keep 64 registers where a thread has two vectors and a row eight
// warps or more, which spills 48 bytes a thread in fp32, 80 with 8 bits out, up to 24 in bf16.
template <typename T>
cudaError_t norm_by_shape(const NormParams& p, cudaStream_t st) {
  const int es = sizeof(T), ys = p.y_dtype == STEP_F32 ? 4 : p.y_dtype <= STEP_F16 ? 2 : 1;
  const bool vec = p.d % 8 == 0 && aligned_to(p.x, p.x_ts, p.x_hs, es, 16) &&
                   (!p.r || (aligned_to(p.r, p.r_ts, p.r_hs, es, 16) && aligned_to(p.sum, p.s_ts, p.s_hs, es, 16))) &&
                   aligned_to(p.w, 0, 0, 1, 16) &&
                   aligned_to(p.y, p.y_ts, p.y_hs, ys, ys == 1 ? 8 : 16);
  const bool many = (long long)p.T * p.H >= 4ll * device_sms();
  if (vec) {
    if (p.d <= 256) return norm_launch<T, 8, 1, 1>(p, st);
    if (p.d <= 2048 && !many) return norm_launch<T, 8, 8, 1>(p, st);
    if (p.d <= 512) return norm_launch<T, 8, 1, 2>(p, st);
    if (p.d <= 1024) return norm_launch<T, 8, 2, 2>(p, st);
    if (p.d <= 2048) return norm_launch<T, 8, 4, 2>(p, st);
    if (p.d <= 4096) return norm_launch<T, 8, 8, 2>(p, st);
    if (p.d <= 8192) return norm_launch<T, 8, 16, 2>(p, st);
    if (p.d <= 16384) return norm_launch<T, 8, 32, 2>(p, st);
    return norm_launch<T, 8, 32, 4>(p, st);
  }
  if (p.d <= 256) return norm_launch<T, 1, 1, 8>(p, st);
  if (p.d <= 2048) return norm_launch<T, 1, 8, 8>(p, st);
  if (p.d <= 8192) return norm_launch<T, 1, 32, 8>(p, st);
  return norm_launch<T, 1, 32, 32>(p, st);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t st) {
  if (p.dtype == STEP_BF16) return norm_by_shape<__nv_bfloat16>(p, st);
  if (p.dtype == STEP_F16) return norm_by_shape<__half>(p, st);
  return norm_by_shape<float>(p, st);
}

}  // namespace moe
