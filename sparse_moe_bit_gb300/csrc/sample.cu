// The next token of rows of logits, with temperature, top-k, top-p and min-p, from a
// given random number (include/step.h).
//
// A row's tokens are ordered by (logit descending, index ascending); every filter keeps a
// first part of that order, so a row's choice is a threshold: a logit, how many tokens of
// that very logit stay (the first by index), and a least weight.  The token is then the
// first whose cumulative kept weight, in order of index, passes u times the total.
//
// Weights w = 2^(-x), x = (max - logit) log2(e) / temperature, are 64-bit integers in
// units of 2^-45 and their sums exact, so that the result depends neither on the order of
// atomics nor on how a row is split.  x is taken in pairs of fp32 numbers (Dekker's
// products and sums), split into a whole number, 1024ths, and a rest r of at most 2^-11;
// 2^(-i/1024) is read from a table, 2^r - 1 is r ln 2 + (r ln 2)^2 / 2 + (r ln 2)^3 / 6.  In
// all a weight is off by 2^-36 of itself; fp32's 2^-22 would put one draw in a few
// hundred of a flat row on the wrong side of a border.
//
// No row is sorted.  A histogram over 1024 bins of x (22 to a factor of two), of counts and
// of mean places within the bin, gives counts exactly and sums of weights to some 1e-3, and
// with them the few bins in which the threshold can lie:
//   top-k    the bin of the k-th token; it and what is above (up to 2048 tokens) go to one
//            CTA of the row, which has all that is left to do
//   top-p    the bins that hold 1 - p of the weights behind them, give or take the
//            histogram's error; one pass sums the weights of all tokens and of those above
//            the band, the band's tokens go to one CTA, which finds the threshold among them
// That CTA sorts the up to 2048 tokens that are left, of a band only those of the 1024th of
// its bins where the weights reach theirs.  Where more are left, the threshold
// comes from histograms over the whole row of the ordered bits (11, 11, 10 of them), of
// counts or of weights, each level among the tokens of the bin before.
//
// Bound: latency for a few rows; for many the chain of a row's steps (read, maximum,
// histogram, its sums over the CTAs, the pass, the threshold, the draw), of which an SM has
// two CTAs' at once where a slice is at most 16400 logits (rows of up to some 131190), else one's;
// and the weights' arithmetic (some 45 instructions an element, once).
// A cluster of up to eight CTAs takes a row: each holds a slice of it in shared memory, read
// from HBM once, and histograms, sums and positions meet through distributed shared memory.
// Measured (fp32 logits, a graph's replay): one row of 130001, top-k 50 and top-p 0.95
// 16.9 us; 48 of 65521 bf16, settings of their own 33; 256 of 131072 (134 MB) greedy 52, no
// filter 141, top-k 50 127, nuclei 240 to 262; of 151936, one CTA an SM, 105, 216, 213 and 444;
// of 131072 where a mask leaves 30 tokens, top-k 50 295, with a nucleus of 0.95 453: fewer
// tokens than k, so that the threshold is -inf, and all levels of the histograms are walked.
// (One CTA a row after another with the next row's read ahead 325, CTAs of 1024 threads 299,
// when this stood at 301.  64 registers, for two CTAs an SM, spill 20 to 24 bytes a thread.)
#include <algorithm>

#include "paged_internal.h"
#include "ptx.cuh"
#include "softmax_df.cuh"
#include "step_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;     // of ordered bits
constexpr int kCoarse = 1024;   // of x
constexpr float kPerOctave = 22.f;
constexpr int kList = 2048;     // tokens that one CTA of a row takes over
constexpr int kNarrow = 256;    // of more, the threshold's 1024th of their bins first (narrow())
constexpr int kOneBit = 45;     // a weight of 1 is 2^45
constexpr unsigned long long kOne = 1ull << kOneBit;

// 2^(-i/32) and 2^(-i/1024), i = 0 .. 31, times 2^63
__device__ const unsigned long long kTable32[32] = {
    0x8000000000000000ull, 0x7d41d96db915019dull, 0x7a92be8a92436616ull, 0x77f25ccdee6d7ae6ull,
    0x75606373ee921c97ull, 0x72dc8373be41a454ull, 0x70666f76154a7089ull, 0x6dfddbcbed791babull,
    0x6ba27e656b4eb57aull, 0x69540ec8f895722dull, 0x6712460a8fc24072ull, 0x64dcdec3371793d1ull,
    0x62b39508aa836d6full, 0x6096266533384a2bull, 0x5e8451cfac061b5full, 0x5c7dd7a3b17dcf75ull,
    0x5a827999fcef3242ull, 0x5891fac0e95612c8ull, 0x56ac1f752150a563ull, 0x54d0ad5a753e077cull,
    0x52ff6b54d8a89c75ull, 0x513821818624b40cull, 0x4f7a993048d088d7ull, 0x4dc69cdceaa72a9cull,
    0x4c1bf828c6dc54b8ull, 0x4a7a77d47f7b84b1ull, 0x48e1e9b9d588e19bull, 0x47521cc5a2e6a9e0ull,
    0x45cae0f1f545eb73ull, 0x444c0740496d4294ull, 0x42d561b3e6243d8aull, 0x4166c34c5615d0ecull};
__device__ const unsigned long long kTable1024[32] = {
    0x8000000000000000ull, 0x7fe9d3a8e07bf086ull, 0x7fd3ab290e46d769ull, 0x7fbd867fdf0acb3bull,
    0x7fa765aca88f6453ull, 0x7f9148aec0b9b7b1ull, 0x7f7b2f857d8c51e5ull, 0x7f651a30352731eeull,
    0x7f4f08ae3dc7c426ull, 0x7f38fafeedc8dd26ull, 0x7f22f1219ba2b4aeull, 0x7f0ceb159deae091ull,
    0x7ef6e8da4b544f9aull, 0x7ee0ea6efaaf4479ull, 0x7ecaefd302e950afull, 0x7eb4f905bb0d4f78ull,
    0x7e9f06067a4360baull, 0x7e8916d497d0e3f4ull, 0x7e732b6f6b18732aull, 0x7e5d43d64b99ddd7ull,
    0x7e47600890f223deull, 0x7e31800592db7078ull, 0x7e1ba3cca92d152cull, 0x7e05cb5d2bdb84beull,
    0x7deff6b672f84e24ull, 0x7dda25d7d6b2177full, 0x7dc458c0af549908ull, 0x7dae8f7055489813ull,
    0x7d98c9e62113e1faull, 0x7d8308216b594720ull, 0x7d6d4a218cd895e5ull, 0x7d578fe5de6e95a0ull};

struct __align__(16) Shared {
  unsigned long long table[1024];  // 2^(-i/1024) in units of 2^-46
  float tablef[1024];              // ... of 2^-41
  union {
    unsigned long long hist[kBins];
    struct {
      uint32_t mine[kCoarse];                   // this CTA's
      uint32_t count[kCoarse], place[kCoarse];  // the row's
    } coarse;
  };
  uint32_t list_key[kList];  // the tokens that this CTA takes over
  int list_at[kList];
  uint16_t local[kList];     // those of its own slice
  unsigned long long warp[kWarps], warp_kept[kWarps], warp_above[kWarps];
  unsigned long long slot[2][3][kMaxCluster];  // totals of the cluster's CTAs, by turns
  unsigned long long found[4];
  float warpf[kWarps];
  uint32_t warpc[kWarps];
  int band[4];
  uint32_t listed, taken;  // tokens of the list; of this CTA's slice
};
static_assert(sizeof(Shared) % 16 == 0, "the slice behind it is written 16 bytes at a time");

// ordered bits: larger numbers have larger keys (of numbers without -0 and NaN)
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
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
__device__ __forceinline__ uint32_t peer_u32(const void* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];"
               : "=r"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ void peer_put(void* p, int rank, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void peer_put32(void* p, int rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t peer_add32(void* p, int rank, uint32_t v) {
  uint32_t r;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;"
               : "=r"(r) : "r"(mapa_shared(smem_u32(p), rank)), "r"(v) : "memory");
  return r;
}
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
// A 64-bit addition as two of 32 bits, which shared memory has (one of 64 is a loop, slow
// where many tokens are alike).
__device__ __forceinline__ void add_wide(unsigned long long* p, unsigned long long v) {
  uint32_t* const w = reinterpret_cast<uint32_t*>(p);
  const uint32_t lo = (uint32_t)v, old = atomicAdd(w, lo);
  const uint32_t hi = (uint32_t)(v >> 32) + (old + lo < old);
  if (hi) atomicAdd(w + 1, hi);
}
template <typename T>
__device__ __forceinline__ T warp_scan(T v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
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
  float max;    // the largest logit
  // a quarter of it, and 4 log2(e) / temperature: a difference of two logits may lie past
  // fp32's end, a quarter of it does not
  float quarter, c_hi, c_lo;
  float bins;   // bins of x for a unit of logits
};
// (No branch: a weight too small to count, of a logit of -inf too, comes out as 0 at x = 47,
// where the correction is at most 2^-10 of the table's, whatever its sum is by then.)
__device__ __forceinline__ unsigned long long weight_of(const Shared& sh, const Row& r, float v) {
  const dflt d = df_two_sum(0.25f * v, -r.quarter);
  const float p = fmaxf(d.hi * r.c_hi, -47.f);  // -x
  const float lo = fmaf(d.hi, r.c_lo, fmaf(d.lo, r.c_hi, fmaf(d.hi, r.c_hi, -p)));
  // the nearest whole number of 1024ths: in the last bits of a sum with 1.5 2^23
  const float t = fmaf(p, 1024.f, 12582912.f);
  const int j = 0x4b400000 - __float_as_int(t);
  const float z = fmaf(t - 12582912.f, -0x1p-10f, p);  // exact
  // 2^(z + lo) - 1
  constexpr float kLn2 = 0x1.62e43p-1f, kLn2Lo = -0x1.05c61p-29f;
  const float y = (z + lo) * kLn2;
  const float q = fmaf(lo, kLn2, fmaf(z, kLn2Lo, y * y * fmaf(y, 0x1.555556p-3f, 0.5f)));
  const float e = fmaf(z, kLn2, q);
  const int i = j & 1023, n = j >> 10;
  // twice the weight, rounded down, and then to the nearest
  const unsigned long long w2 = sh.table[i] + (unsigned long long)((long long)__float2int_rn(sh.tablef[i] * e) << 5);
  const unsigned long long w = ((w2 >> n) + 1) >> 1;
  return v == r.max ? kOne : w;
}
// where x lies among the bins (monotone in v)
__device__ __forceinline__ float place_of(const Row& r, float v) {
  return fminf(v == r.max ? 0.f : (r.max - v) * r.bins, (float)(kCoarse - 1));
}

// Tokens to look at: a CTA's slice of the row, or the list that one CTA has taken over.
struct View {
  const float* v;         // (list: nullptr)
  const uint32_t* key;
  const int* at;
  int n, begin, chunk;    // chunk: of a warp, contiguous
  int cluster, rank;
  __device__ __forceinline__ uint32_t key_at(int i) const { return v ? key_of(v[i]) : key[i]; }
  __device__ __forceinline__ int index(int i) const { return v ? begin + i : at[i]; }
  __device__ __forceinline__ void sync() const {
    if (cluster > 1) cluster_sync(); else __syncthreads();
  }
};

// A row's CTA: the steps that several of its paths share.
struct Worker {
  Shared& sh;
  const Row& r;
  const int tid, lane, warp;
  int turn = 1;  // of sh.slot: two sets, so that one may still be read while the other is written

  // the sums over the cluster's CTAs: before this one, and of all
  __device__ void totals(const View& w, unsigned long long mine, unsigned long long& before,
                         unsigned long long& all) {
    if (tid < w.cluster) peer_put(&sh.slot[turn][0][w.rank], tid, mine);
    w.sync();
    before = all = 0;
    for (int c = 0; c < w.cluster; ++c) {
      const unsigned long long x = sh.slot[turn][0][c];
      if (c < w.rank) before += x;
      all += x;
    }
    turn ^= 1;
  }

  // The key at which the sum over (key descending) of 1 (counts) or of weights reaches
  // `target`; `above` gets the sum over larger keys, `here` that of the key itself.  Weights:
  // of keys above `low` alone, whose own tokens count as `tie` together.
  __device__ uint32_t select(const View& w, bool mass, unsigned long long target, uint32_t low,
                             unsigned long long tie, unsigned long long& above, unsigned long long& here) {
    const int w0 = min(warp * w.chunk, w.n), w1 = min(w0 + w.chunk, w.n);
    uint32_t prefix = 0;
    above = 0;
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
      __syncthreads();
      for (int i = w0 + lane; i < w1; i += 32) {
        const uint32_t key = w.key_at(i);
        if (level > 0 && key >> (shift + bits) != prefix) continue;
        const int bin = key >> shift & ((1u << bits) - 1);
        if (!mass) atomicAdd(reinterpret_cast<uint32_t*>(&sh.hist[bin]), 1u);
        else if (key > low) add_wide(&sh.hist[bin], weight_of(sh, r, value_of(key)));
      }
      if (mass && tie && w.rank == 0 && tid == 0 && (level == 0 || low >> (shift + bits) == prefix))
        add_wide(&sh.hist[low >> shift & ((1u << bits) - 1)], tie);
      w.sync();
      // this CTA's share of the bins, over the cluster, largest first
      const int share = kBins / w.cluster, b0 = kBins - 1 - w.rank * share;
      const int each = max(share / kThreads, 1);
      const bool has = tid < share;
      unsigned long long v[kBins / kThreads], sum = 0;
#pragma unroll
      for (int e = 0; e < kBins / kThreads; ++e) {
        v[e] = 0;
        if (has && e < each)
          for (int c = 0; c < w.cluster; ++c) v[e] += peer_u64(&sh.hist[b0 - tid * each - e], w.cluster > 1 ? c : w.rank);
        sum += v[e];
      }
      const unsigned long long inc = warp_scan(sum, lane);
      if (lane == 31) sh.warp[warp] = inc;
      __syncthreads();
      unsigned long long before = 0, all = 0, less, whole;
      for (int x = 0; x < kWarps; ++x) {
        if (x < warp) before += sh.warp[x];
        all += sh.warp[x];
      }
      totals(w, all, less, whole);
      unsigned long long at = above + less + before + inc - sum;
      if (has) {
#pragma unroll
        for (int e = 0; e < kBins / kThreads; ++e) {
          if (e < each && at < target && target <= at + v[e]) {
            for (int c = 0; c < w.cluster; ++c) {
              peer_put(&sh.found[0], w.cluster > 1 ? c : w.rank, at);
              peer_put(&sh.found[1], w.cluster > 1 ? c : w.rank, v[e]);
              peer_put(&sh.found[2], w.cluster > 1 ? c : w.rank, (unsigned long long)(b0 - tid * each - e));
            }
          }
          at += v[e];
        }
      }
      w.sync();
      above = sh.found[0];
      here = sh.found[1];
      prefix = prefix << bits | (uint32_t)sh.found[2];
    }
    return prefix;
  }

  // sums of f over the warps' chunks, into `out`
  template <typename F>
  __device__ void chunk_sums(const View& w, F f, unsigned long long* out) {
    const int w0 = min(warp * w.chunk, w.n), w1 = min(w0 + w.chunk, w.n);
    unsigned long long sum = 0;
    for (int i = w0 + lane; i < w1; i += 32) sum += f(w.key_at(i), w.index(i));
    sum = warp_sum(sum);
    __syncthreads();  // (out may still be read)
    if (lane == 0) out[warp] = sum;
    __syncthreads();
  }

  // The first token at which the sum of f(key, index), in order of index, passes
  // `target(total)`, where `sums` are the warps' sums: the thread that has it calls
  // found(index, total, f there).
  template <typename F, typename G, typename H>
  __device__ void locate(const View& w, F f, G target_of, const unsigned long long* sums, H found) {
    unsigned long long all = 0, at, total;
    for (int x = 0; x < kWarps; ++x) all += sums[x];
    totals(w, all, at, total);
    const unsigned long long target = target_of(total);
    if (at <= target && target < at + all) {  // here: which warp's chunk, then which token
      int x = 0;
      while (at + sums[x] <= target) at += sums[x++];
      __syncthreads();
      const int c0 = min(x * w.chunk, w.n), c1 = min(c0 + w.chunk, w.n);
      const int each = (c1 - c0 + kThreads - 1) / kThreads;
      const int i0 = min(c0 + tid * each, c1), i1 = min(i0 + each, c1);
      unsigned long long mine = 0;
      for (int i = i0; i < i1; ++i) mine += f(w.key_at(i), w.index(i));
      const unsigned long long inc = warp_scan(mine, lane);
      if (lane == 31) sh.warp[warp] = inc;
      __syncthreads();
      for (int y = 0; y < warp; ++y) at += sh.warp[y];
      at += inc - mine;
      if (at <= target && target < at + mine) {
        for (int i = i0; i < i1; ++i) {
          const unsigned long long v = f(w.key_at(i), w.index(i));
          if (target < at + v) {
            found(w.index(i), total, v);
            break;
          }
          at += v;
        }
      }
    }
  }
};

// Sorts size <= E kThreads numbers (a power of two of at least 32 E; thread t has those at
// E t .. E t + E - 1), largest first: bitonic, within a thread, a warp, or through `s`.
template <int E>
__device__ __forceinline__ void sort(unsigned long long (&v)[E], int size, unsigned long long* s) {
  const int i0 = threadIdx.x * E;
  for (int m = 2; m <= size; m *= 2) {
    for (int d = m / 2; d > 0; d /= 2) {
      if (d < E) {
#pragma unroll
        for (int b = 1; b < E; b *= 2) {
          if (b != d) continue;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (e & b) continue;
            const unsigned long long x = v[e], y = v[e | b];
            const bool swap = (x < y) == (((i0 + e) & m) == 0);
            v[e] = swap ? y : x;
            v[e | b] = swap ? x : y;
          }
        }
      } else if (d < 32 * E) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const unsigned long long x = v[e], y = __shfl_xor_sync(0xffffffffu, x, d / E);
          const bool larger = (((i0 + e) & d) == 0) == (((i0 + e) & m) == 0);
          v[e] = larger == (x > y) ? x : y;
        }
      } else {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) s[i0 + e] = v[e];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const unsigned long long x = v[e], y = s[(i0 + e) ^ d];
          const bool larger = (((i0 + e) & d) == 0) == (((i0 + e) & m) == 0);
          v[e] = larger == (x > y) ? x : y;
        }
      }
    }
  }
}
__device__ __forceinline__ int sort_size(int n, int E) {
  int size = 32 * E;
  while (size < n) size *= 2;
  return size;
}

// The sums over the CTA of what the threads before have, and of all.
__device__ __forceinline__ void block_scan(Shared& sh, unsigned long long mine, unsigned long long& before,
                                           unsigned long long& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned long long inc = warp_scan(mine, lane);
  __syncthreads();
  if (lane == 31) sh.warp[warp] = inc;
  __syncthreads();
  before = inc - mine;
  all = 0;
#pragma unroll
  for (int x = 0; x < kWarps; ++x) {
    if (x < warp) before += sh.warp[x];
    all += sh.warp[x];
  }
}

// The filters over the up to kList tokens of a view that one CTA has: sorted by (key
// descending, index ascending).  total: the weights that top_p is a part of (0: those of the
// first k tokens here); above: of tokens that are not here, larger than all.  False where the
// threshold does not lie here.
template <int E>
__device__ bool settle_n(Shared& sh, const Row& r, const View& w, int k, float top_p, unsigned long long total,
                         unsigned long long above, uint32_t& thr, int& cut) {
  const int tid = threadIdx.x;
  unsigned long long* s = sh.hist;
  unsigned long long key[E], v[E], sum = 0, at, all;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = tid * E + e;
    key[e] = i < w.n ? (unsigned long long)w.key_at(i) << 32 | (uint32_t)~w.index(i) : 0ull;
  }
  sort<E>(key, sort_size(w.n, E), s);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = tid * E + e;
    v[e] = i < w.n && (k == 0 || i < k) ? weight_of(sh, r, value_of((uint32_t)(key[e] >> 32))) : 0ull;
    sum += v[e];
  }
  block_scan(sh, sum, at, all);
  if (total == 0) total = all;
  unsigned long long target = ~0ull;
  if (top_p < 1.f) {
    target = max(times<true>(total, top_p), 1ull);
    if (target <= above || target > above + all) return false;  // (the same in all threads)
    target -= above;
  }
  // the last token that stays has weight, begins before the target, and the next does not
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const unsigned long long next = at + v[e];
    if (v[e] > 0 && at < target && (next >= target || next == all)) sh.found[0] = key[e];
    at = next;
  }
  __syncthreads();
  thr = (uint32_t)(sh.found[0] >> 32);
  cut = (int)~(uint32_t)sh.found[0];
  return true;
}
__device__ bool settle(Shared& sh, const Row& r, const View& w, int k, float top_p, unsigned long long total,
                       unsigned long long above, uint32_t& thr, int& cut) {
  __syncthreads();
  static_assert(kList == 4 * kThreads, "tokens of a thread");
  if (w.n <= kThreads) return settle_n<1>(sh, r, w, k, top_p, total, above, thr, cut);
  if (w.n <= 2 * kThreads) return settle_n<2>(sh, r, w, k, top_p, total, above, thr, cut);
  return settle_n<4>(sh, r, w, k, top_p, total, above, thr, cut);
}

// Of a list of tokens in bins `first_bin` .. `last_bin`, those of the 1024th of that span in
// which the weights reach `target`, where they do; `above` is with the weights before it.
// (Sorting 2000 tokens takes some 12 us, this and a sort of what is left 3: 256 rows of
// 131072, nucleus of 0.99 at temperature 2, 353 -> 308 us then; where lists are short there is
// nothing in it, and from 64 tokens on a loss: 48 rows of settings of their own 35 -> 38.)
__device__ void narrow(Shared& sh, const Row& r, View& w, int first_bin, int last_bin, unsigned long long target,
                       unsigned long long& above) {
  constexpr int E = kList / kThreads, FINE = 2 * kThreads;
  const int tid = threadIdx.x;
  const float scale = (float)FINE / (float)(last_bin + 1 - first_bin);
  uint32_t key[E];
  int at[E], bin[E];
  for (int i = tid; i < FINE; i += kThreads) sh.hist[i] = 0;
  if (tid == 0) sh.listed = 0;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = e * kThreads + tid;
    bin[e] = -1;
    if (i < w.n) {
      key[e] = w.key[i];
      at[e] = w.at[i];
      const float v = value_of(key[e]);
      bin[e] = min(max((int)((place_of(r, v) - (float)first_bin) * scale), 0), FINE - 1);
      add_wide(&sh.hist[bin[e]], weight_of(sh, r, v));
    }
  }
  __syncthreads();
  const unsigned long long h0 = sh.hist[2 * tid], h1 = sh.hist[2 * tid + 1];
  unsigned long long before, all;
  block_scan(sh, h0 + h1, before, all);
  if (target <= above || target > above + all) return;  // (the same in all threads)
  before += above;
  if (before < target && target <= before + h0 + h1) {
    const bool second = before + h0 < target;
    sh.found[0] = second ? before + h0 : before;
    sh.found[1] = 2 * tid + second;
  }
  __syncthreads();
  above = sh.found[0];
  const int which = (int)sh.found[1];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (bin[e] != which) continue;
    const uint32_t to = atomicAdd(&sh.listed, 1u);  // (no further than where all have been read)
    sh.list_key[to] = key[e];
    sh.list_at[to] = at[e];
  }
  __syncthreads();
  w.n = (int)sh.listed;
}

// what is kept: tokens above `thr`, of its own the ones up to index `cut`, and none of a
// weight below `least`
struct Kept {
  uint32_t thr;
  int cut;
  unsigned long long least;
};

// The draw among the tokens of a list (in any order) that are kept.
template <int E, typename Put>
__device__ void draw_n(Shared& sh, const Row& r, const View& w, const Kept& keep, float u, Put put) {
  const int tid = threadIdx.x;
  unsigned long long key[E], v[E], sum = 0, at, total;
#pragma unroll
  for (int e = 0; e < E; ++e) {  // by index, the first first
    const int i = tid * E + e;
    key[e] = i < w.n ? (unsigned long long)(uint32_t)~w.index(i) << 32 | (uint32_t)i : 0ull;
  }
  sort<E>(key, sort_size(w.n, E), sh.hist);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    v[e] = 0;
    if (tid * E + e < w.n) {
      const int i = (int)(uint32_t)key[e];
      const uint32_t k = w.key_at(i);
      if (k > keep.thr || (k == keep.thr && w.index(i) <= keep.cut)) {
        const unsigned long long x = weight_of(sh, r, value_of(k));
        v[e] = x >= keep.least ? x : 0;
      }
    }
    sum += v[e];
  }
  block_scan(sh, sum, at, total);
  const unsigned long long target = times<false>(total, u);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (at <= target && target < at + v[e]) put((int)~(uint32_t)(key[e] >> 32), total, v[e]);
    at += v[e];
  }
}
template <typename Put>
__device__ void draw_sorted(Shared& sh, const Row& r, const View& w, const Kept& keep, float u, Put put) {
  if (w.n <= kThreads) draw_n<1>(sh, r, w, keep, u, put);
  else draw_n<kList / kThreads>(sh, r, w, keep, u, put);
}

template <typename T>
__device__ __forceinline__ float logit_of(uint32_t bits) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(bits);
  else if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((uint16_t)bits));
  else return __uint_as_float(bits << 16);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleParams p, int cluster,
                                                          int slice) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  float* vals = reinterpret_cast<float*>(smem + sizeof(Shared));
  const int row = blockIdx.x / cluster, rank = blockIdx.x % cluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // (shared memory of another CTA is there once that has begun: waited for below)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  // The slices begin at 16-byte boundaries of memory: the first one's up to VEC - 1 places
  // before the row are filled with -inf, which no filter ever draws from.
  constexpr int VEC = 16 / sizeof(T);
  const T* const src = static_cast<const T*>(p.logits) + row * p.stride;
  const int begin = rank * slice - (int)(reinterpret_cast<uintptr_t>(src) / sizeof(T) % VEC);
  const int n = max(min(p.V - begin, slice), 0);
  const int chunk = (slice + kThreads - 1) / kThreads * 32;
  const int w0 = min(warp * chunk, n), w1 = min(w0 + chunk, n);

  const float temperature = p.temperature ? p.temperature[row] : p.all_temperature;
  const bool greedy = !(temperature > 0.f);
  int k = p.top_k ? p.top_k[row] : p.all_top_k;
  if (k <= 0 || k >= p.V) k = 0;
  float top_p = p.top_p ? p.top_p[row] : p.all_top_p;
  if (!(top_p < 1.f)) top_p = 1.f;
  top_p = fmaxf(top_p, 0.f);
  float min_p = p.min_p ? p.min_p[row] : p.all_min_p;
  if (!(min_p > 0.f)) min_p = 0.f;
  min_p = fminf(min_p, 1.f);
  float u = p.u[row];
  if (!(u > 0.f)) u = 0.f;
  u = fminf(u, 0x1.fffffep-1f);

  // ---- the slice into shared memory, the largest logit and its first index
  // vectors of a thread in flight (four times as many, which fp32 registers cannot hold
  // beside the rest: 256 x 131072 267 us for 255, one row of 130001 18.7 for 16.9)
  constexpr int AHEAD = 8 / VEC;
  const int vecs = (n + VEC - 1) / VEC;
  auto load = [&](int i, uint4& v) {
    const int at = begin + i * VEC;
    if (at >= 0 && at + VEC <= p.V) {
      v = __ldg(reinterpret_cast<const uint4*>(src + at));
    } else {
      uint32_t u[4] = {0, 0, 0, 0};
      for (int e = 0; e < VEC; ++e) {
        uint32_t bits = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;
        if (at + e >= 0 && at + e < p.V) {
          if constexpr (sizeof(T) == 4) bits = __float_as_uint(src[at + e]);
          else bits = reinterpret_cast<const uint16_t*>(src)[at + e];
        }
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (w == e * 4 / VEC) u[w] |= sizeof(T) == 4 ? bits : bits << (16 * (e & 1));
      }
      v = make_uint4(u[0], u[1], u[2], u[3]);
    }
  };
  uint4 ahead[AHEAD];
#pragma unroll
  for (int j = 0; j < AHEAD; ++j)
    if (tid + j * kThreads < vecs) load(tid + j * kThreads, ahead[j]);
  for (int i = tid; i < 1024; i += kThreads) {
    const unsigned long long t = __umul64hi(kTable32[i >> 5], kTable1024[i & 31]);  // 2^62 x
    sh.tablef[i] = (float)t * 0x1p-21f;
    sh.table[i] = (t + (1ull << (60 - kOneBit))) >> (61 - kOneBit);
  }
  float best = -INFINITY;
  int best_at = 0x7fffffff;
  for (int base = tid; base < vecs; base += AHEAD * kThreads) {
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int i = base + j * kThreads;
      if (i >= vecs) break;
      const uint32_t u[4] = {ahead[j].x, ahead[j].y, ahead[j].z, ahead[j].w};
      if (i + AHEAD * kThreads < vecs) load(i + AHEAD * kThreads, ahead[j]);
      float x[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        x[e] = logit_of<T>(sizeof(T) == 4 ? u[e & 3] : u[e / 2 & 3] >> (16 * (e & 1)) & 0xffffu);
        x[e] = x[e] == x[e] ? x[e] + 0.f : -INFINITY;  // (-0 is +0)
        if (x[e] > best) {
          best = x[e];
          best_at = begin + i * VEC + e;
        }
      }
#pragma unroll
      for (int e = 0; e < VEC; e += 4)
        *reinterpret_cast<float4*>(vals + i * VEC + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    }
  }
  unsigned long long first = (unsigned long long)key_of(best) << 32 | (uint32_t)~best_at;
#pragma unroll
  for (int d = 16; d; d >>= 1) first = max(first, __shfl_xor_sync(0xffffffffu, first, d));
  if (lane == 0) sh.warp[warp] = first;
  if (tid == 0) sh.listed = sh.taken = 0;
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (tid < cluster) {
    unsigned long long m = 0;
    for (int w = 0; w < kWarps; ++w) m = max(m, sh.warp[w]);
    peer_put(&sh.slot[0][0][rank], tid, m);
  }
  cluster_sync();
  first = 0;
  for (int c = 0; c < cluster; ++c) first = max(first, sh.slot[0][0][c]);
  const bool none = (uint32_t)(first >> 32) <= kLowest;
  if (greedy || none) {
    if (rank == 0 && tid == 0) {
      p.token[row] = none ? -1 : (int)~(uint32_t)first;
      if (p.logprob) p.logprob[row] = none ? __int_as_float(0x7fffffff) : 0.f;
    }
    return;
  }
  Row r;
  r.max = value_of((uint32_t)(first >> 32));
  r.quarter = 0.25f * r.max;
  {
    // (fp64 costs microseconds here)
    const dflt c = df_div(dflt{4 * 0x1.715476p+0f, 4 * 0x1.4ae0cp-26f}, dflt{temperature, 0.f});
    const bool finite = c.hi < INFINITY;  // (else one of 0, or past fp32's end)
    r.c_hi = finite ? c.hi : temperature < 1.f ? INFINITY : 0.f;
    r.c_lo = finite ? c.lo : 0.f;
    r.bins = fminf(0.25f * r.c_hi * kPerOctave, 1e38f);
  }
  Worker work{sh, r, tid, lane, warp};
  const View whole{vals, nullptr, nullptr, n, begin, chunk, cluster, rank};
  Kept keep{kLowest, -1, 1};  // (nothing at -inf)
  if (min_p > 0.f) keep.least = max(times<true>(kOne, min_p), 1ull);
  auto kept_weight = [&](uint32_t key, int at) -> unsigned long long {
    if (key < keep.thr || (key == keep.thr && at > keep.cut)) return 0;
    const unsigned long long w = weight_of(sh, r, value_of(key));
    return w >= keep.least ? w : 0;
  };
  auto draw = [u](unsigned long long total) { return times<false>(total, u); };
  auto put = [&](int token, unsigned long long total, unsigned long long value) {
    p.token[row] = token;
    if (p.logprob) {
      const unsigned long long rest = total - value;
      p.logprob[row] = rest < value ? log1pf(-((float)rest / (float)total)) : logf((float)value / (float)total);
    }
  };
  // the filters over the tokens of a view, all of which they concern
  auto filter = [&](const View& w) {
    unsigned long long equal = 0, of_equal = 0, above;  // tokens of the threshold's key; how many stay
    bool cut = false;
    if (k > 0) {
      keep.thr = work.select(w, false, k, 0, 0, above, equal);
      of_equal = k - above;
      cut = true;
    }
    if (top_p < 1.f) {
      const unsigned long long tie = k > 0 ? of_equal * weight_of(sh, r, value_of(keep.thr)) : 0;
      unsigned long long here, all = 0, before, total;
      const uint32_t low = keep.thr;
      work.chunk_sums(w, [&](uint32_t key, int) { return key > low ? weight_of(sh, r, value_of(key)) : 0ull; }, sh.warp);
      for (int x = 0; x < kWarps; ++x) all += sh.warp[x];
      work.totals(w, all, before, total);
      const unsigned long long target = max(times<true>(total + tie, top_p), 1ull);
      const uint32_t thr = work.select(w, true, target, low, tie, above, here);
      const unsigned long long one = weight_of(sh, r, value_of(thr));
      if (thr != low || k == 0) equal = here / one;
      of_equal = (target - above + one - 1) / one;
      keep.thr = thr;
      cut = true;
    }
    if (cut) {
      keep.cut = 0x7fffffff;
      if (of_equal < equal) {
        const uint32_t thr = keep.thr;
        auto is = [thr](uint32_t key, int) -> unsigned long long { return key == thr; };
        work.chunk_sums(w, is, sh.warp_kept);
        work.locate(w, is, [of_equal](unsigned long long) { return of_equal - 1; }, sh.warp_kept,
                    [&](int i, unsigned long long, unsigned long long) {
                      for (int c = 0; c < w.cluster; ++c)
                        peer_put(&sh.found[0], w.cluster > 1 ? c : w.rank, (unsigned long long)i);
                    });
        w.sync();
        keep.cut = (int)sh.found[0];
      }
    }
  };

  if (p.V + VEC > kList && (k > 0 || top_p < 1.f)) {
    // ---- counts and mean places in the bins of x: a token is 2^place_bits + its place in
    // the bin, in as many of its leading bits as the sums of a slice leave room for
    auto& co = sh.coarse;
    const int count_bits = 32 - __clz(slice), level_bits = max(32 - 2 * count_bits, 0);
    const int place_bits = level_bits ? count_bits + level_bits : 0;
    const float levels = (float)(1 << level_bits);
    for (int i = tid; i < kCoarse; i += kThreads) co.mine[i] = 0;
    __syncthreads();
    if (k > 0 && k <= kThreads * cluster / 4) {
      // of the threads' largest logits alone: the bin up to which there are k of those holds
      // no fewer than k of all tokens, and few more
      if (best > -INFINITY) atomicAdd(&co.mine[(int)place_of(r, best)], 1u << place_bits);
    } else {
#pragma unroll 4
      for (int i = w0 + lane; i < w1; i += 32) {
        const float x = place_of(r, vals[i]);
        const int b = (int)x;
        atomicAdd(&co.mine[b], level_bits ? (1u << place_bits) + (uint32_t)((x - (float)b) * levels) : 1u);
      }
    }
    cluster_sync();
    {
      const int share = kCoarse / cluster;
      for (int i = tid; i < share; i += kThreads) {
        const int b = rank * share + i;
        uint32_t v[kMaxCluster], count = 0, place = 0;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) v[c] = c < cluster ? peer_u32(&co.mine[b], c) : 0;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          count += v[c] >> place_bits;
          if (level_bits) place += v[c] & ((1u << place_bits) - 1);
        }
        for (int c = 0; c < cluster; ++c) {
          peer_put32(&co.count[b], c, count);
          peer_put32(&co.place[b], c, place);
        }
      }
    }
    cluster_sync();
    // ---- which bins: two a thread
    const int b0 = 2 * tid;
    const uint32_t n0 = co.count[b0], n1 = co.count[b0 + 1];
    const uint32_t inc = warp_scan(n0 + n1, lane);
    if (lane == 31) sh.warpc[warp] = inc;
    if (tid < 4) sh.band[tid] = kCoarse;  // first bin, last bin, tokens above the first, up to the last
    __syncthreads();
    uint32_t upto = inc - n0 - n1;
    for (int x = 0; x < warp; ++x) upto += sh.warpc[x];
    const uint32_t c0 = upto + n0, c1 = c0 + n1;  // tokens up to either bin
    if (k > 0) {
      for (int e = 0; e < 2; ++e) {
        const uint32_t before = e ? c0 : upto, after = e ? c1 : c0;
        if (before < (uint32_t)k && (uint32_t)k <= after) {
          sh.band[0] = 0;
          sh.band[1] = b0 + e;
          sh.band[2] = 0;
          sh.band[3] = (int)after;
        }
      }
      __syncthreads();
    } else {
      // weights: the bin's at its edge, less the mean place's part of the bin's span;
      // summed from the far end, so that small sums keep their bits
      constexpr float kSpan = 0.031015526f;  // 1 - 2^(-1/22)
      auto mass = [&](int b, uint32_t count) {
        if (count == 0 || b == kCoarse - 1) return 0.f;
        // (a level stands for its middle)
        const float places = ((float)co.place[b] + 0.5f * (float)count) / levels;
        return exp2f(-(float)b * (1.f / kPerOctave)) * ((float)count - places * kSpan);
      };
      const float m0 = mass(b0, n0), m1 = mass(b0 + 1, n1);
      float suffix = m0 + m1;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const float o = __shfl_down_sync(0xffffffffu, suffix, d);
        if (lane + d < 32) suffix += o;
      }
      if (lane == 0) sh.warpf[warp] = suffix;
      float after = __shfl_down_sync(0xffffffffu, suffix, 1);
      if (lane == 31) after = 0.f;
      __syncthreads();
      float sum = 0.f;
      for (int x = kWarps - 1; x >= 0; --x) {
        if (x > warp) after += sh.warpf[x];
        sum += sh.warpf[x];
      }
      // the first bins behind which there is surely no more, and surely less, than the rest
      const float rest = (1.f - top_p) * sum;
      // (half a level, 1.3e-4 for the chord of 2^(-x) over a bin, fp32's sums)
      const float off = 2.f * (kSpan * 0.5f / levels + 5e-4f);
      const float hi = rest * (1.f + off) + 1e-6f * sum, lo = rest * (1.f - off) - 1e-6f * sum;
      for (int e = 0; e < 2; ++e) {
        const float s = e ? after : after + m1;  // behind bin b0 + e
        if (s <= hi) atomicMin(&sh.band[0], b0 + e);
        if (s <= lo) atomicMin(&sh.band[1], b0 + e);
      }
      __syncthreads();
      for (int e = 0; e < 2; ++e) {
        if (sh.band[0] == b0 + e) sh.band[2] = (int)(e ? c0 : upto);
        if (sh.band[1] == b0 + e) sh.band[3] = (int)(e ? c1 : c0);
      }
      __syncthreads();
    }
    const int first_bin = sh.band[0], last_bin = sh.band[1];
    const bool fits = first_bin <= last_bin && last_bin < kCoarse && sh.band[3] - sh.band[2] <= kList;
    if (fits) {  // (the same in all CTAs of the row, which hold the same sums)
      // ---- one pass: the band's tokens go to the row's first CTA, in any order; top-p:
      // weights of all tokens, of those above the band, and of those that min-p leaves of them
      unsigned long long sum = 0, above = 0, kept = 0;
      auto take = [&](int i, float v) {
        const uint32_t mine = atomicAdd(&sh.taken, 1u);
        if (mine < (uint32_t)kList) sh.local[mine] = (uint16_t)i;
        const uint32_t at = peer_add32(&sh.listed, 0, 1);
        if (at < (uint32_t)kList) {
          peer_put32(&sh.list_key[at], 0, key_of(v));
          peer_put32(&sh.list_at[at], 0, (uint32_t)(begin + i));
        }
      };
      if (k > 0) {
#pragma unroll 4
        for (int i = w0 + lane; i < w1; i += 32) {
          const float v = vals[i];
          if ((int)place_of(r, v) <= last_bin) take(i, v);
        }
      } else {
        // (places against the band's borders as numbers: floor is monotone)
        const float first_place = (float)first_bin, end_place = (float)(last_bin + 1);
        auto pass = [&](auto minimum) {
#pragma unroll 4
          for (int i = w0 + lane; i < w1; i += 32) {
            const float v = vals[i], x = place_of(r, v);
            const unsigned long long w = weight_of(sh, r, v);
            sum += w;
            above += x < first_place ? w : 0;
            if (minimum()) kept += x < first_place && w >= keep.least ? w : 0;
            if (x >= first_place && x < end_place) take(i, v);
          }
        };
        if (keep.least > 1) {
          pass([] { return true; });
        } else {
          pass([] { return false; });
          kept = above;
        }
        sum = warp_sum(sum);
        above = warp_sum(above);
        kept = warp_sum(kept);
        if (lane == 0) {
          sh.warp[warp] = sum;
          sh.warp_above[warp] = above;
          sh.warp_kept[warp] = kept;
        }
      }
      __syncthreads();
      unsigned long long mine[3] = {sh.taken, 0, 0};
      if (k == 0) {
        for (int x = 0; x < kWarps; ++x) {
          mine[1] += sh.warp[x];
          mine[2] += sh.warp_above[x];
        }
      }
      if (tid < cluster)
#pragma unroll
        for (int e = 0; e < 3; ++e) peer_put(&sh.slot[work.turn][e][rank], tid, mine[e]);
      cluster_sync();
      unsigned long long got[3] = {0, 0, 0};
      for (int c = 0; c < cluster; ++c)
#pragma unroll
        for (int e = 0; e < 3; ++e) got[e] += sh.slot[work.turn][e][c];
      work.turn ^= 1;
      const int listed = (int)got[0];
      const View list{nullptr, sh.list_key, sh.list_at, listed, 0, 0, 1, 0};
      if (listed <= kList && k > 0) {  // all that is left is in the list
        if (rank != 0) return;
        settle(sh, r, list, k, top_p, 0, 0, keep.thr, keep.cut);
        draw_sorted(sh, r, list, keep, u, put);
        return;
      }
      if (listed <= kList) {
        if (rank == 0) {
          View left = list;
          if (listed > kNarrow)
            narrow(sh, r, left, first_bin, last_bin, max(times<true>(got[1], top_p), 1ull), got[2]);
          const bool good = settle(sh, r, left, 0, top_p, got[1], got[2], keep.thr, keep.cut);
          if (tid < cluster) {
            peer_put(&sh.found[2], tid, good ? keep.thr : 0ull);
            peer_put(&sh.found[3], tid, (unsigned long long)(uint32_t)keep.cut);
          }
        }
        cluster_sync();
        if (sh.found[2] != 0) {
          keep.thr = (uint32_t)sh.found[2];
          keep.cut = (int)(uint32_t)sh.found[3];
          // the band's tokens that stay join their chunks' sums
          for (int i = tid; i < (int)mine[0]; i += kThreads) {
            const int at = sh.local[i];
            const unsigned long long w = kept_weight(key_of(vals[at]), begin + at);
            if (w) add_wide(&sh.warp_kept[at / chunk], w);
          }
          __syncthreads();
          work.locate(whole, kept_weight, draw, sh.warp_kept, put);
          return;
        }
        keep.thr = kLowest;
        keep.cut = -1;
        cluster_sync();
      }
    }
  }
  if (k > 0 || top_p < 1.f) {
    if (p.V + VEC <= kList) settle(sh, r, whole, k, top_p, 0, 0, keep.thr, keep.cut);
    else filter(whole);
    work.chunk_sums(whole, kept_weight, sh.warp_kept);
  } else {
    unsigned long long sum = 0;
#pragma unroll 4
    for (int i = w0 + lane; i < w1; i += 32) {
      const unsigned long long w = weight_of(sh, r, vals[i]);
      sum += w >= keep.least ? w : 0;
    }
    sum = warp_sum(sum);
    if (lane == 0) sh.warp_kept[warp] = sum;
    __syncthreads();
  }
  work.locate(whole, kept_weight, draw, sh.warp_kept, put);
}

template <typename T>
cudaError_t sample_launch(const SampleParams& p, cudaStream_t st) {
  // CTAs of a row: until two fit an SM (256 rows, top-p 0.9: of 40000 logits 4 CTAs of a row 90
  // us, 2 that have an SM each 99; 49152 100 and 111; 98304 8 CTAs 216, 4 226; 70000 184 and 181,
  // with L2 cold 196 and 200), and while they are no more than run at once with half as many for
  // each (48 rows of 65521: 8 CTAs each 34 us, although the last rows wait for the first; 4
  // each 39)
  constexpr int kOfSm = 228 * 1024, kOfCta = 1024;  // shared memory; what a CTA takes beside its own
  const int sms = device_sms();
  // (the row may begin up to seven places behind a 16-byte boundary)
  auto slice_of = [&](int c) { return ((p.V + 7 + c - 1) / c + 7) / 8 * 8; };
  auto bytes_of = [&](int c) { return (int)sizeof(Shared) + slice_of(c) * 4; };
  int cluster = 1;
  while (cluster < kMaxCluster && (2 * (bytes_of(cluster) + kOfCta) > kOfSm ||
                                   (p.V > 2048 * cluster && (long long)p.B * cluster < 2 * sms)))
    cluster *= 2;
  const int slice = slice_of(cluster), smem = bytes_of(cluster);
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
