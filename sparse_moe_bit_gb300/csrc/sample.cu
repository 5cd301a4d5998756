// The next token of rows of logits, with temperature, top-k, top-p and min-p, from a
// given random number (include/step.h).
//
// A row's tokens are ordered by (logit descending, index ascending); every filter keeps a
// first part of that order, so a row's choice is a threshold: a key, how many tokens of
// that very key stay (the first by index), and a least weight.  No sort: the threshold
// comes from histograms of the keys' bits (11, 11, 10 of them), of counts for top-k and of
// weights for top-p, each level among the keys of the bin before.  The token is then the
// first whose cumulative kept weight, in order of index, passes u times the total.
//
// Weights w = 2^(-x), x = (max - logit) log2(e) / temperature, are 64-bit integers in
// units of 2^-45 and their sums exact, so that the result depends neither on the order of
// atomics nor on how a row is split.  x is taken in pairs of fp32 numbers (Dekker's
// products and sums), split into a whole number, 1024ths, and a rest r below 2^-11;
// 2^(-i/1024) is read from a table, 2^r - 1 is r ln 2 + (r ln 2)^2 / 2 + (r ln 2)^3 / 6.  In
// all a weight is off by 2^-36 of itself; fp32's 2^-22 would put one draw in a few
// hundred of a flat row on the wrong side of a border.
//
// Bound: latency for a few rows, HBM (and the weights' arithmetic, some 40 operations
// an element) for many.  A cluster of up to eight CTAs takes a row: each holds a slice of
// its keys in shared memory, read from HBM once, and histograms, sums and positions meet
// through distributed shared memory.
#include <algorithm>

#include "paged_internal.h"
#include "ptx.cuh"
#include "softmax_df.cuh"
#include "step_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kOneBit = 45;  // a weight of 1 is 2^45
constexpr unsigned long long kOne = 1ull << kOneBit;

// 2^(-i/32) and 2^(-i/1024), i = 0 .. 31, times 2^63
__device__ const unsigned long long kCoarse[32] = {
    0x8000000000000000ull, 0x7d41d96db915019dull, 0x7a92be8a92436616ull, 0x77f25ccdee6d7ae6ull,
    0x75606373ee921c97ull, 0x72dc8373be41a454ull, 0x70666f76154a7089ull, 0x6dfddbcbed791babull,
    0x6ba27e656b4eb57aull, 0x69540ec8f895722dull, 0x6712460a8fc24072ull, 0x64dcdec3371793d1ull,
    0x62b39508aa836d6full, 0x6096266533384a2bull, 0x5e8451cfac061b5full, 0x5c7dd7a3b17dcf75ull,
    0x5a827999fcef3242ull, 0x5891fac0e95612c8ull, 0x56ac1f752150a563ull, 0x54d0ad5a753e077cull,
    0x52ff6b54d8a89c75ull, 0x513821818624b40cull, 0x4f7a993048d088d7ull, 0x4dc69cdceaa72a9cull,
    0x4c1bf828c6dc54b8ull, 0x4a7a77d47f7b84b1ull, 0x48e1e9b9d588e19bull, 0x47521cc5a2e6a9e0ull,
    0x45cae0f1f545eb73ull, 0x444c0740496d4294ull, 0x42d561b3e6243d8aull, 0x4166c34c5615d0ecull};
__device__ const unsigned long long kFine[32] = {
    0x8000000000000000ull, 0x7fe9d3a8e07bf086ull, 0x7fd3ab290e46d769ull, 0x7fbd867fdf0acb3bull,
    0x7fa765aca88f6453ull, 0x7f9148aec0b9b7b1ull, 0x7f7b2f857d8c51e5ull, 0x7f651a30352731eeull,
    0x7f4f08ae3dc7c426ull, 0x7f38fafeedc8dd26ull, 0x7f22f1219ba2b4aeull, 0x7f0ceb159deae091ull,
    0x7ef6e8da4b544f9aull, 0x7ee0ea6efaaf4479ull, 0x7ecaefd302e950afull, 0x7eb4f905bb0d4f78ull,
    0x7e9f06067a4360baull, 0x7e8916d497d0e3f4ull, 0x7e732b6f6b18732aull, 0x7e5d43d64b99ddd7ull,
    0x7e47600890f223deull, 0x7e31800592db7078ull, 0x7e1ba3cca92d152cull, 0x7e05cb5d2bdb84beull,
    0x7deff6b672f84e24ull, 0x7dda25d7d6b2177full, 0x7dc458c0af549908ull, 0x7dae8f7055489813ull,
    0x7d98c9e62113e1faull, 0x7d8308216b594720ull, 0x7d6d4a218cd895e5ull, 0x7d578fe5de6e95a0ull};

struct Shared {
  unsigned long long table[1024];  // 2^(-i/1024) in units of 2^-45
  float tablef[1024];
  unsigned long long hist[kBins];
  unsigned long long warp[kWarps + 1];
  unsigned long long slot[2][kMaxCluster];  // totals of the cluster's CTAs, by turns
  unsigned long long found[4];
  uint32_t best[kMaxCluster][2];
};

// ordered bits: larger numbers have larger keys; -0 is +0, NaN is -inf
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!(x == x)) x = -INFINITY;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
constexpr uint32_t kLowest = 0x007fffffu;  // key_of(-inf)

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned long long peer_u64(const void* p, int rank) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];"
               : "=l"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ void peer_put(void* p, int rank, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), rank)), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
// x * f rounded down (UP: up), for 0 <= f <= 1
template <bool UP>
__device__ __forceinline__ unsigned long long times(unsigned long long x, float f) {
  if (f >= 1.f) return x;
  const uint32_t b = __float_as_uint(f);
  const int e = (int)(b >> 23);                      // f = m 2^(max(e, 1) - 150)
  const unsigned long long m = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int s = 150 - (e ? e : 1);                   // 24 .. 149
  unsigned long long lo = x * m, hi = __umul64hi(x, m);
  if (s >= 128) return UP && (lo | hi) ? 1 : 0;
  unsigned long long r, rest;
  if (s >= 64) {
    r = s == 64 ? hi : hi >> (s - 64);
    rest = (s == 64 ? 0 : hi << (128 - s)) | lo;
  } else {
    r = (lo >> s) | (hi << (64 - s));
    rest = lo << (64 - s);
  }
  return r + (UP && rest ? 1 : 0);
}

struct Row {
  uint32_t top;         // the largest key
  // a quarter of its logit, and 4 log2(e) / temperature: a difference of two logits may
  // lie past fp32's end, a quarter of it does not
  float max, c_hi, c_lo;
};
__device__ __forceinline__ unsigned long long weight_of(const Shared& sh, const Row& r, uint32_t key) {
  if (key == r.top) return kOne;
  const dflt d = df_two_sum(0.25f * value_of(key), -r.max);
  const float p = d.hi * r.c_hi;  // -x
  if (!(p > -46.f)) return 0;
  const float lo = fmaf(d.hi, r.c_lo, fmaf(d.lo, r.c_hi, fmaf(d.hi, r.c_hi, -p)));
  const float jn = rintf(p * 1024.f);
  const float z = fmaf(jn, -0x1p-10f, p);  // exact
  const int j = -(int)jn;
  // 2^(z + lo) - 1
  constexpr float kLn2 = 0x1.62e43p-1f, kLn2Lo = -0x1.05c61p-29f;
  const float y = (z + lo) * kLn2;
  const float q = fmaf(lo, kLn2, fmaf(z, kLn2Lo, y * y * fmaf(y, 0x1.555556p-3f, 0.5f)));
  const float e = fmaf(z, kLn2, q);
  const int i = j & 1023, n = j >> 10;
  const long long add = (long long)__float2int_rn(sh.tablef[i] * e * 0x1p41f) << 4;
  return (sh.table[i] + add + (1ull << n >> 1)) >> n;
}

// the row's kept tokens: those above `thr`, of its own the ones up to index `cut`, and none
// of a weight below `least`
struct Kept {
  uint32_t thr;
  int cut;
  unsigned long long least;
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleParams p, int cluster,
                                                          int slice) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + sizeof(Shared));
  const int row = blockIdx.x / cluster, rank = blockIdx.x % cluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int begin = rank * slice, n = max(min(p.V - begin, slice), 0);
  const int chunk = (slice + kThreads - 1) / kThreads * 32;  // of a warp: contiguous
  const int w0 = min(warp * chunk, n), w1 = min(w0 + chunk, n);

  float temperature = p.temperature ? p.temperature[row] : 1.f;
  const bool greedy = !(temperature > 0.f);
  int k = p.top_k ? p.top_k[row] : 0;
  if (k <= 0 || k >= p.V) k = 0;
  float top_p = p.top_p ? p.top_p[row] : 1.f;
  if (!(top_p < 1.f)) top_p = 1.f;
  top_p = fmaxf(top_p, 0.f);
  float min_p = p.min_p ? p.min_p[row] : 0.f;
  if (!(min_p > 0.f)) min_p = 0.f;
  min_p = fminf(min_p, 1.f);
  float u = p.u[row];
  if (!(u > 0.f)) u = 0.f;
  u = fminf(u, 0x1.fffffep-1f);

  // ---- keys into shared memory, the largest and its first index
  uint32_t best = 0;
  int best_at = 0x7fffffff;
  {
    const T* src = static_cast<const T*>(p.logits) + row * p.stride + begin;
#pragma unroll 8
    for (int i = w0 + lane; i < w1; i += 32) {
      float x;
      if constexpr (sizeof(T) == 4) x = src[i];
      else if constexpr (std::is_same<T, __half>::value) x = __half2float(src[i]);
      else x = __bfloat162float(src[i]);
      const uint32_t key = key_of(x);
      keys[i] = key;
      if (key > best) {
        best = key;
        best_at = begin + i;
      }
    }
  }
  for (int i = tid; i < 1024; i += kThreads) {
    const unsigned long long t = __umul64hi(kCoarse[i >> 5], kFine[i & 31]);  // 2^62 x
    sh.tablef[i] = (float)t * 0x1p-62f;
    sh.table[i] = (t + (1ull << (61 - kOneBit))) >> (62 - kOneBit);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const uint32_t o = __shfl_xor_sync(0xffffffffu, best, d);
    const int at = __shfl_xor_sync(0xffffffffu, best_at, d);
    if (o > best || (o == best && at < best_at)) best = o, best_at = at;
  }
  if (lane == 0) sh.warp[warp] = (unsigned long long)best << 32 | (uint32_t)~best_at;
  __syncthreads();
  if (tid == 0) {
    unsigned long long m = 0;
    for (int w = 0; w < kWarps; ++w) m = max(m, sh.warp[w]);
    for (int c = 0; c < cluster; ++c) peer_put(&sh.slot[0][rank], c, m);
  }
  cluster_sync();
  unsigned long long first = 0;
  for (int c = 0; c < cluster; ++c) first = max(first, sh.slot[0][c]);
  Row r;
  r.top = (uint32_t)(first >> 32);
  r.max = 0.25f * value_of(r.top);
  int turn = 1;  // of sh.slot: two sets, so that one may still be read while the other is written

  if (greedy || r.top <= kLowest) {
    if (rank == 0 && tid == 0) {
      const bool none = r.top <= kLowest;
      p.token[row] = none ? -1 : (int)~(uint32_t)first;
      if (p.logprob) p.logprob[row] = none ? __int_as_float(0x7fffffff) : 0.f;
    }
    cluster_sync();
    return;
  }
  {
    const double c = 4 * 1.4426950408889634 / (double)temperature;
    r.c_hi = (float)c;
    r.c_lo = r.c_hi < INFINITY ? (float)(c - (double)r.c_hi) : 0.f;
  }

  // The key at which the sum over (key descending) of 1 (counts) or of weights reaches
  // `target`; `above` gets the sum over larger keys, `here` that of the key itself.  Of the
  // weights, tokens of key `tie` count as `tie_n` together.
  auto select = [&](bool mass, unsigned long long target, uint32_t low, unsigned long long tie_weight,
                    unsigned long long& above, unsigned long long& here) -> uint32_t {
    uint32_t prefix = 0;
    above = 0;
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
      __syncthreads();
      for (int i = w0 + lane; i < w1; i += 32) {
        const uint32_t key = keys[i];
        if (level > 0 && key >> (shift + bits) != prefix) continue;
        const int bin = key >> shift & ((1u << bits) - 1);
        if (!mass) atomicAdd(reinterpret_cast<uint32_t*>(&sh.hist[bin]), 1u);
        else if (key > low) atomicAdd(&sh.hist[bin], weight_of(sh, r, key));
      }
      if (mass && tie_weight && rank == 0 && tid == 0 && (level == 0 || low >> (shift + bits) == prefix))
        atomicAdd(&sh.hist[low >> shift & ((1u << bits) - 1)], tie_weight);
      cluster_sync();
      // this CTA's share of the bins, over the cluster, largest first
      const int share = kBins / cluster, b0 = kBins - 1 - rank * share;
      unsigned long long v[kBins / kThreads], sum = 0;
      const int each = max(share / kThreads, 1);
      const bool has = tid < share;
      for (int e = 0; e < each; ++e) {
        v[e] = 0;
        if (has)
          for (int c = 0; c < cluster; ++c) v[e] += peer_u64(&sh.hist[b0 - tid * each - e], c);
        sum += v[e];
      }
      unsigned long long inc = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      if (lane == 31) sh.warp[warp] = inc;
      __syncthreads();
      unsigned long long before = 0, all = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sh.warp[w];
        all += sh.warp[w];
      }
      if (tid < cluster) peer_put(&sh.slot[turn][rank], tid, all);
      cluster_sync();
      unsigned long long at = above + before + inc - sum;
      for (int c = 0; c < rank; ++c) at += sh.slot[turn][c];
      turn ^= 1;
      if (has) {
        for (int e = 0; e < each; ++e) {
          if (at < target && target <= at + v[e]) {
            for (int c = 0; c < cluster; ++c) {
              peer_put(&sh.found[0], c, at);
              peer_put(&sh.found[1], c, v[e]);
              peer_put(&sh.found[2], c, (unsigned long long)(b0 - tid * each - e));
            }
          }
          at += v[e];
        }
      }
      cluster_sync();
      above = sh.found[0];
      here = sh.found[1];
      prefix = prefix << bits | (uint32_t)sh.found[2];
    }
    return prefix;
  };

  // The first index at which the sum of f(key, index) passes `target(total)`; total and
  // f there are returned, in every CTA.
  auto locate = [&](auto f, auto target_of, unsigned long long& total, unsigned long long& value) -> int {
    unsigned long long sum = 0;
    for (int i = w0 + lane; i < w1; i += 32) sum += f(keys[i], begin + i);
    sum = warp_sum(sum);
    __syncthreads();  // (sh.warp may still be read)
    if (lane == 0) sh.warp[warp] = sum;
    __syncthreads();
    unsigned long long all = 0;
    for (int w = 0; w < kWarps; ++w) all += sh.warp[w];
    if (tid < cluster) peer_put(&sh.slot[turn][rank], tid, all);
    cluster_sync();
    unsigned long long at = 0;
    total = 0;
    for (int c = 0; c < cluster; ++c) {
      if (c < rank) at += sh.slot[turn][c];
      total += sh.slot[turn][c];
    }
    turn ^= 1;
    const unsigned long long target = target_of(total);
    if (at <= target && target < at + all) {  // here: which warp's chunk, then which token
      int w = 0;
      while (at + sh.warp[w] <= target) at += sh.warp[w++];
      __syncthreads();
      const int c0 = min(w * chunk, n), c1 = min(c0 + chunk, n);
      const int each = (c1 - c0 + kThreads - 1) / kThreads;
      const int i0 = min(c0 + tid * each, c1), i1 = min(i0 + each, c1);
      unsigned long long mine = 0;
      for (int i = i0; i < i1; ++i) mine += f(keys[i], begin + i);
      unsigned long long inc = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      if (lane == 31) sh.warp[warp] = inc;
      __syncthreads();
      for (int x = 0; x < warp; ++x) at += sh.warp[x];
      at += inc - mine;
      if (at <= target && target < at + mine) {
        for (int i = i0; i < i1; ++i) {
          const unsigned long long v = f(keys[i], begin + i);
          if (target < at + v) {
            for (int c = 0; c < cluster; ++c) {
              peer_put(&sh.found[0], c, (unsigned long long)(begin + i));
              peer_put(&sh.found[1], c, v);
            }
            break;
          }
          at += v;
        }
      }
    }
    cluster_sync();
    value = sh.found[1];
    return (int)sh.found[0];
  };

  Kept keep{kLowest, -1, 1};  // (nothing at -inf)
  unsigned long long equal = 0, of_equal = 0;  // tokens of the threshold's key; how many stay
  if (k > 0) {
    unsigned long long above;
    keep.thr = select(false, k, 0, 0, above, equal);
    of_equal = k - above;
  }
  if (top_p < 1.f) {
    const unsigned long long w_thr = k > 0 ? weight_of(sh, r, keep.thr) : 0, tie = of_equal * w_thr;
    unsigned long long total, value, above, here;
    // (the kept tokens' weights)
    {
      unsigned long long sum = 0;
      for (int i = w0 + lane; i < w1; i += 32)
        if (keys[i] > keep.thr) sum += weight_of(sh, r, keys[i]);
      sum = warp_sum(sum);
      __syncthreads();
      if (lane == 0) sh.warp[warp] = sum;
      __syncthreads();
      unsigned long long all = 0;
      for (int w = 0; w < kWarps; ++w) all += sh.warp[w];
      if (tid < cluster) peer_put(&sh.slot[turn][rank], tid, all);
      cluster_sync();
      total = tie;
      for (int c = 0; c < cluster; ++c) total += sh.slot[turn][c];
      turn ^= 1;
    }
    (void)value;
    const unsigned long long target = max(times<true>(total, top_p), 1ull);
    const uint32_t thr = select(true, target, keep.thr, tie, above, here);
    const unsigned long long w = weight_of(sh, r, thr);
    if (thr != keep.thr) equal = here / w;
    of_equal = (target - above + w - 1) / w;
    keep.thr = thr;
  }
  if (min_p > 0.f) keep.least = max(times<true>(kOne, min_p), 1ull);
  if (k > 0 || top_p < 1.f) {
    keep.cut = 0x7fffffff;
    if (of_equal < equal) {
      unsigned long long total, value;
      const uint32_t thr = keep.thr;
      keep.cut = locate([thr](uint32_t key, int) -> unsigned long long { return key == thr; },
                        [of_equal](unsigned long long) { return of_equal - 1; }, total, value);
      cluster_sync();  // (sh.found is read before it is written again)
    }
  }
  unsigned long long total, value;
  const int token = locate(
      [&](uint32_t key, int at) -> unsigned long long {
        if (key < keep.thr || (key == keep.thr && at > keep.cut)) return 0;
        const unsigned long long w = weight_of(sh, r, key);
        return w >= keep.least ? w : 0;
      },
      [u](unsigned long long total) { return times<false>(total, u); }, total, value);
  if (rank == 0 && tid == 0) {
    p.token[row] = token;
    if (p.logprob) {
      const unsigned long long rest = total - value;
      p.logprob[row] = rest < value ? log1pf(-((float)rest / (float)total)) : logf((float)value / (float)total);
    }
  }
}

template <typename T>
cudaError_t sample_launch(const SampleParams& p, cudaStream_t st) {
  const int sms = device_sms();
  int cluster = 1;
  while (cluster < kMaxCluster && (p.V > 24576 * cluster || (p.V > 2048 * cluster && (long long)p.B * cluster < 2 * sms)))
    cluster *= 2;
  const int slice = (p.V + cluster - 1) / cluster;
  const int smem = (int)sizeof(Shared) + slice * 4;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem((const void*)sample_kernel<T>, 232448 - 1024, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(p.B * cluster));
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = cluster;
  a[0].val.clusterDim.y = 1;
  a[0].val.clusterDim.z = 1;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, sample_kernel<T>, p, cluster, slice);
}

}  // namespace

cudaError_t launch_sample(const SampleParams& p, cudaStream_t st) {
  if (p.dtype == STEP_F32) return sample_launch<float>(p, st);
  if (p.dtype == STEP_F16) return sample_launch<__half>(p, st);
  return sample_launch<__nv_bfloat16>(p, st);
}

}  // namespace moe
