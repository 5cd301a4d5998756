// Maintenance of a paged cache (include/paged.h): fork, reserve, free and
// compact change the integer state, pages_copy moves the pages' rows.
//
// The state is small (a few hundred kilobytes at most) and the calls are
// latency-bound.  fork and free are independent per pair or slot: one CTA
// each, the counts of shared pages by integer atomics, whose order does not
// change a sum.  reserve and compact number things across the whole state: one
// CTA of 1024 threads that runs block-wide prefix sums over it, four pages a
// thread and step -- "the k-th free page" is then the page whose exclusive
// prefix is k, so the lowest numbers are taken first whatever the threads'
// timing, and no list of free pages has to be kept.  pages_copy is bound by
// HBM: 16 KB pieces, each thread four 16-byte loads before its stores.  Measured:
// 900 pages in 20 pools, 64 KB each, 370 us, 6.4 TB/s of reads and writes (0.95 of
// the copy rate, 28 registers).
#include "paged_internal.h"

namespace moe {
namespace {

constexpr int kScanThreads = 1024;

// Inclusive prefix sum of two 32-bit counters (packed) over the block;
// returns the inclusive value, *total the block's sum.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* total, uint64_t* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();  // sh of the previous call is read
  if (lane == 31) sh[warp] = v;
  __syncthreads();
  if (warp == 0) {
    uint64_t w = sh[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint64_t o = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += o;
    }
    sh[32 + lane] = w;
  }
  __syncthreads();
  *total = sh[63];
  return v + (warp ? sh[32 + warp - 1] : 0);
}

__global__ void __launch_bounds__(128) fork_kernel(int32_t* refs, int P, int32_t* table,
                                                   long long ts, int width, int32_t* lens, int S,
                                                   const int32_t* src, const int32_t* dst, int F,
                                                   int32_t* refused) {
  const int i = blockIdx.x;
  const int s = src[i], d = dst[i];
  bool bad = s < 0 || s >= S || d < 0 || d >= S;
  // an earlier pair with the same dst, or a pair whose dst is this src
  for (int j = threadIdx.x; j < F; j += blockDim.x) {
    const int e = dst[j];
    if (e == s || (j < i && e == d)) bad = true;
  }
  bad = __syncthreads_or(bad);
  const int len = bad ? 0 : lens[s];
  if (!bad && lens[d] != 0) bad = true;
  // every thread has read lens before it changes (no other CTA writes lens[d]
  // unless it has the same dst, and then this one is the earliest or refused)
  __syncthreads();
  if (bad) {
    if (threadIdx.x == 0 && refused) atomicAdd(refused, 1);
    return;
  }
  const int32_t* row = table + (long long)s * ts;
  int32_t* out = table + (long long)d * ts;
  for (int c = threadIdx.x; c < width; c += blockDim.x) {
    const int pg = row[c];
    out[c] = pg;
    if (pg >= 0 && pg < P) atomicAdd(refs + pg, 1);
  }
  if (threadIdx.x == 0) lens[d] = len;
}

__global__ void __launch_bounds__(128) free_kernel(int32_t* refs, int P, int32_t* table,
                                                   long long ts, int width, int32_t* lens, int S,
                                                   const int32_t* slots, int F) {
  const int i = blockIdx.x;
  const int s = slots[i];
  bool bad = s < 0 || s >= S;
  for (int j = threadIdx.x; j < i; j += blockDim.x)
    if (slots[j] == s) bad = true;
  if (__syncthreads_or(bad)) return;
  int32_t* row = table + (long long)s * ts;
  for (int c = threadIdx.x; c < width; c += blockDim.x) {
    const int pg = row[c];
    if (pg >= 0 && pg < P) atomicSub(refs + pg, 1);
    row[c] = -1;
  }
  if (threadIdx.x == 0) lens[s] = 0;
}

struct Need {
  int have, want, own;  // pages held, pages wanted, 1: the last one is exchanged
  int last;             // the page exchanged
  bool narrow;          // the table's row is too short
};
__device__ __forceinline__ Need need_of(int s, const int32_t* refs, int P, const int32_t* table,
                                        long long ts, int width, const int32_t* lens,
                                        const int32_t* add, int page) {
  Need n;
  const long long len = max(lens[s], 0), more = max(add[s], 0);
  n.have = (int)((len + page - 1) / page);
  const long long want = (len + more + page - 1) / page;
  n.narrow = more > 0 && (want > width || len + more > 0x7fffffff);  // (lens is int32)
  n.want = n.narrow ? n.have : (int)want;
  n.own = 0;
  n.last = -1;
  if (more > 0 && len % page != 0 && n.have <= width) {
    n.last = table[(long long)s * ts + n.have - 1];
    n.own = n.last >= 0 && n.last < P && refs[n.last] > 1;
  }
  return n;
}

__global__ void __launch_bounds__(kScanThreads) reserve_kernel(
    int32_t* refs, int P, int32_t* table, long long ts, int width, int32_t* lens,
    const int32_t* add, int S, int page, int32_t* moves, int32_t* status, int32_t* first) {
  __shared__ uint64_t sh[64];
  const int tid = threadIdx.x;
  // first[s]: pages taken by the slots before s; counts of narrow slots beside
  uint64_t base = 0;
  for (int s0 = 0; s0 < S; s0 += kScanThreads) {
    const int s = s0 + tid;
    uint64_t v = 0, total;
    int mine = 0;
    if (s < S) {
      const Need n = need_of(s, refs, P, table, ts, width, lens, add, page);
      mine = n.want - n.have + n.own;
      v = (uint64_t)(uint32_t)mine | ((uint64_t)n.narrow << 32);
    }
    const uint64_t inc = block_scan(v, &total, sh) + base;
    if (s < S) {
      first[s] = (int)(uint32_t)inc - mine;
      moves[2 * s] = -1;
      moves[2 * s + 1] = -1;
    }
    base += total;
  }
  const int needed = (int)(uint32_t)base, narrow = (int)(base >> 32);
  if (tid == 0) first[S] = needed;
  // free pages
  int nfree = 0;
  {
    uint64_t mine = 0, total;
    for (int p = tid; p < P; p += kScanThreads) mine += refs[p] == 0;
    block_scan(mine, &total, sh);
    nfree = (int)total;
  }
  const int missing = max(needed - nfree, 0);
  if (tid == 0) {
    status[0] = missing;
    status[1] = narrow;
  }
  if (missing || narrow) return;
  __syncthreads();  // first[] and moves[] written by all
  // The k-th free page goes to the slot s with first[s] <= k < first[s + 1].
  // refs is read (all of a step) before it is written (none but pages of this
  // step, and only free ones become used).
  int taken = 0;
  for (int p0 = 0; p0 < P && taken < needed; p0 += kScanThreads * 4) {
    const int p = p0 + tid * 4;
    int free4 = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (p + j < P && refs[p + j] == 0) free4 |= 1 << j;
    uint64_t total;
    int k = (int)block_scan((uint64_t)__popc(free4), &total, sh) - __popc(free4) + taken;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!(free4 >> j & 1)) continue;
      if (k < needed) {
        int lo = 0, hi = S;  // first[lo] <= k < first[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (first[mid] <= k) lo = mid; else hi = mid;
        }
        const int s = lo, at = k - first[s];
        const long long len = max(lens[s], 0), more = max(add[s], 0);
        const int have = (int)((len + page - 1) / page);
        const int cnt = first[s + 1] - first[s];
        const int fresh = (int)((len + more + page - 1) / page) - have;
        const int own = cnt - fresh;  // 1: the slot's first page replaces its last
        if (own && at == 0) {
          moves[2 * s] = table[(long long)s * ts + have - 1];
          moves[2 * s + 1] = p + j;
        }
        table[(long long)s * ts + have - own + at] = p + j;
        refs[p + j] = 1;
      }
      ++k;
    }
    taken += (int)total;
  }
  __syncthreads();
  for (int s = tid; s < S; s += kScanThreads) {
    const int old = moves[2 * s];
    if (old >= 0) atomicSub(refs + old, 1);
    lens[s] = max(lens[s], 0) + max(add[s], 0);
  }
}

__global__ void __launch_bounds__(kScanThreads) compact_plan_kernel(int32_t* refs, int P,
                                                                    int32_t* moves, int32_t* count,
                                                                    int32_t* to) {
  __shared__ uint64_t sh[64];
  const int tid = threadIdx.x;
  uint64_t mine = 0, total;
  for (int p = tid; p < P; p += kScanThreads) mine += refs[p] > 0;
  block_scan(mine, &total, sh);
  const int live = (int)total;
  // counters packed: free numbers below `live` (low), pages in use above (high)
  uint64_t base = 0;
  for (int p0 = 0; p0 < P; p0 += kScanThreads * 4) {
    const int p = p0 + tid * 4;
    uint32_t used = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (p + j < P && refs[p + j] > 0) used |= 1u << j;
    uint64_t v = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (p + j >= P) break;
      const bool u = used >> j & 1;
      if (!u && p + j < live) v += 1;
      if (u && p + j >= live) v += 1ull << 32;
    }
    uint64_t k = block_scan(v, &total, sh) - v + base;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (p + j >= P) break;
      const bool u = used >> j & 1;
      if (!u && p + j < live) {
        moves[2 * (int)(uint32_t)k + 1] = p + j;
        k += 1;
      }
      if (u && p + j >= live) {
        moves[2 * (int)(k >> 32)] = p + j;
        k += 1ull << 32;
      }
      if (!u && p + j >= live) to[p + j] = -1;  // a stale number in a table stays
    }
    base += total;
  }
  const int n = (int)(uint32_t)base;  // as many as (base >> 32)
  __syncthreads();
  for (int i = tid; i < P; i += kScanThreads) {
    if (i < n) {
      const int a = moves[2 * i], b = moves[2 * i + 1];
      refs[b] = refs[a];
      to[a] = b;
    } else {
      moves[2 * i] = -1;
      moves[2 * i + 1] = -1;
    }
  }
  __syncthreads();
  for (int i = tid; i < n; i += kScanThreads) refs[moves[2 * i]] = 0;
  if (tid == 0) {
    *count = n;
    // pages below `live` keep their numbers: the remap needs no entry there
    to[P] = live;
  }
}

__global__ void __launch_bounds__(256) compact_table_kernel(int32_t* table, long long ts, int width,
                                                            int S, int P, const int32_t* to) {
  const int live = to[P];
  const long long n = (long long)S * width;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long s = i / width;
    int32_t* e = table + s * ts + (i - s * width);
    const int pg = *e;
    if (pg >= live && pg < P) {
      const int q = to[pg];
      if (q >= 0) *e = q;
    }
  }
}

constexpr int kCopyThreads = 256;
constexpr int kCopyPiece = kCopyThreads * 16 * 4;  // bytes a CTA moves a step

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(uint8_t* pools, int B,
                                                            long long pool_stride, int P,
                                                            long long page_stride,
                                                            long long page_bytes,
                                                            const int32_t* moves, int M,
                                                            const int32_t* count, int pieces) {
  const int m = count ? min(max(*count, 0), M) : M;
  const long long units = (long long)m * B * pieces;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int i = (int)(u / ((long long)B * pieces));
    const long long rest = u - (long long)i * B * pieces;
    const int b = (int)(rest / pieces), piece = (int)(rest - (long long)b * pieces);
    const int from = moves[2 * i], to = moves[2 * i + 1];
    if (from < 0 || from >= P || to < 0 || to >= P || from == to) continue;
    const uint8_t* src = pools + b * pool_stride + from * page_stride;
    uint8_t* dst = pools + b * pool_stride + to * page_stride;
    const long long at = (long long)piece * kCopyPiece + threadIdx.x * 16;
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (at + j * kCopyThreads * 16 < page_bytes)
        v[j] = __ldcs(reinterpret_cast<const uint4*>(src + at + j * kCopyThreads * 16));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (at + j * kCopyThreads * 16 < page_bytes)
        *reinterpret_cast<uint4*>(dst + at + j * kCopyThreads * 16) = v[j];
  }
}

}  // namespace

cudaError_t launch_pages_fork(int32_t* refs, int P, int32_t* table, long long ts, int width,
                              int32_t* lens, int S, const int32_t* src, const int32_t* dst, int F,
                              int32_t* refused, cudaStream_t st) {
  return launch_kernel(fork_kernel, dim3(F), dim3(128), 0, st, refs, P, table, ts, width, lens, S,
                       src, dst, F, refused);
}

cudaError_t launch_pages_reserve(int32_t* refs, int P, int32_t* table, long long ts, int width,
                                 int32_t* lens, const int32_t* add, int S, int page,
                                 int32_t* moves, int32_t* status, int32_t* scratch,
                                 cudaStream_t st) {
  return launch_kernel(reserve_kernel, dim3(1), dim3(kScanThreads), 0, st, refs, P, table, ts,
                       width, lens, add, S, page, moves, status, scratch);
}

cudaError_t launch_pages_free(int32_t* refs, int P, int32_t* table, long long ts, int width,
                              int32_t* lens, int S, const int32_t* slots, int F, cudaStream_t st) {
  return launch_kernel(free_kernel, dim3(F), dim3(128), 0, st, refs, P, table, ts, width, lens, S,
                       slots, F);
}

cudaError_t launch_pages_compact(int32_t* refs, int P, int32_t* table, long long ts, int width,
                                 int S, int32_t* moves, int32_t* count, int32_t* scratch,
                                 cudaStream_t st) {
  cudaError_t e = launch_kernel(compact_plan_kernel, dim3(1), dim3(kScanThreads), 0, st, refs, P,
                                moves, count, scratch);
  if (e != cudaSuccess) return e;
  const long long n = (long long)S * width;
  if (n == 0) return cudaSuccess;
  const long long want = (n + 1023) / 1024;
  const int cap = device_sms() * 4;
  return launch_kernel(compact_table_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(256),
                       0, st, table, ts, width, S, P, (const int32_t*)scratch);
}

cudaError_t launch_pages_copy(uint8_t* pools, int B, long long pool_stride, int P,
                              long long page_stride, long long page_bytes, const int32_t* moves,
                              int M, const int32_t* count, cudaStream_t st) {
  const int pieces = (int)((page_bytes + kCopyPiece - 1) / kCopyPiece);
  const long long units = (long long)M * B * pieces;
  const long long cap = (long long)device_sms() * 8;
  return launch_kernel(copy_kernel, dim3((unsigned)(units < cap ? units : cap)),
                       dim3(kCopyThreads), 0, st, pools, B, pool_stride, P, page_stride,
                       page_bytes, moves, M, count, pieces);
}

}  // namespace moe
