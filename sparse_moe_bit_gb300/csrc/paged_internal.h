// Internal structures of the paged-cache operators (include/paged.h).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "moe_internal.h"
#include "paged.h"

namespace moe {

// n / d for 0 <= n < 2^31 by one multiplication: mul = ceil(2^(31+s) / d) with
// 2^s >= d, whose excess over the exact reciprocal stays below one part in
// 2^31 of a unit.
struct FastDiv {
  uint32_t mul = 0;
  int shift = 0;
  int d = 1;
};
inline FastDiv make_fastdiv(int d) {
  FastDiv f;
  f.d = d;
  int s = 0;
  while ((1ll << s) < d) ++s;
  f.shift = 31 + s;
  f.mul = (uint32_t)(((1ull << f.shift) + (uint64_t)d - 1) / (uint64_t)d);
  return f;
}
__device__ __forceinline__ int fast_div(int n, const FastDiv& f) {
  return (int)(((uint64_t)(uint32_t)n * f.mul) >> f.shift);
}

struct CacheView {
  uint16_t* k;
  uint16_t* v;
  int pages, page, heads, dim;
  long long page_stride, row_stride, head_stride;
  FastDiv div;  // by page
};

struct BatchView {
  const int32_t* table;
  const int32_t* cu;
  const int32_t* kv_len;
  int N, T, width;
  long long table_stride;
  int capacity;  // min(width * page, 2^31 - 1): the longest context a table row holds
};

// One sequence of a batch with its metadata made safe.
struct Seq {
  int t0, nq, kv;  // first new token, new tokens, context
};
__device__ __forceinline__ Seq load_seq(const BatchView& b, int n) {
  Seq s;
  const int t0 = min(max(b.cu[n], 0), b.T);
  const int t1 = min(max(b.cu[n + 1], t0), b.T);
  s.t0 = t0;
  s.nq = t1 - t0;
  s.kv = min(max(b.kv_len[n], 0), b.capacity);
  return s;
}
// The sequence of new token t: the last n with cu[n] <= t (-1: none).
__device__ __forceinline__ int find_seq(const BatchView& b, int t) {
  int lo = -1, hi = b.N;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// ---- rotary positions (rope.cu)
struct RopeParams {
  // plain: x -> out [T][H][D]; append: x = q -> out, plus k, v -> cache
  const void* x;
  void* out;
  int T, H, D;
  long long x_ts, x_hs, o_ts, o_hs;
  const int32_t* pos;  // plain only
  const double* freq;
  int r;
  float mscale, sign;
  bool interleaved, in_place;
  // append
  const void* k;
  const void* v;
  long long k_ts, v_ts;
  CacheView c;
  BatchView b;
  int* err;
  // set by the launch: tokens of a CTA, divisions
  int tokens;
  FastDiv div_r, div_tok, div_q, div_k, div_v;
};
cudaError_t launch_rope(const RopeParams& p, int dtype, bool append, cudaStream_t st);

// ---- attention over the paged cache
struct AttnParams {
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  long long q_ts, q_hs, o_ts, o_hs;
  int Hq, G;       // query heads; query heads of a key/value head
  FastDiv divG;
  CacheView c;
  BatchView b;
  float scale_log2;  // scale * log2(e)
  int causal, window;
  // 256-row tiles: `tiles` of the batch; chunk c of a tile covers the keys
  // [c, c+1) * chunk behind its first visible one, the last goes to the end.
  // Partial results [T * Hq][chunks] where chunks > 1.
  int tiles, chunks, chunk;
  // tiles of `row_tile` = 8 or 16 rows: `warps` (a multiple of kRowWarps) share the
  // work; partial results [2 * warps][16], groups of keys before each sequence
  // [N + 1].
  int warps, row_tile;
  int parts;  // about so many partial results of a row
  long long* before;
  float* part_o;    // [..][D], unnormalised
  float2* part_ml;  // [..]: running maximum (log2 units) and sum
  int* err;
};
// The first key in a query's window.  (A query before position 0 sees none; its
// position less a window near 2^31 would not fit.)
__device__ __forceinline__ int window_begin(int pos, int window) { return max(pos, 0) - window + 1; }
// the first and one past the last key that rows [r0, r1) of a sequence see
// (r1 > r0; row r is new token r / G)
__device__ __forceinline__ int2 key_range(const AttnParams& p, const Seq& s, int r0, int r1) {
  const int p0 = s.kv - s.nq + fast_div(r0, p.divG);
  const int p1 = s.kv - s.nq + fast_div(r1 - 1, p.divG);
  int lo = 0, hi = s.kv;
  if (p.causal) hi = min(hi, p1 + 1);
  if (p.window > 0) lo = max(0, window_begin(p0, p.window));
  return make_int2(lo, max(hi, lo));
}
// A tensor map over one of the cache's arrays (innermost first: feature, row of a
// page, head, page): boxes of `box` rows of a page x `features` (64: 128-byte
// swizzle, 32: 64-byte), zero fill out of bounds; false where the array has none
// (a stride that the encoding refuses).  (paged_api.cu)
bool make_page_map(CUtensorMap* m, const void* base, const CacheView& c, int features, int box,
                   bool bf16);
// Log2 of the largest softmax weight that is rounded to the 16-bit type.  fp16 holds
// 2^15 and rounds off by up to 2^-25 whatever is small: with weights up to 1 a key 17.4
// nats behind the largest would vanish, and a long tail of such keys with it
// (one-sidedly, while the sums count them).  bf16 has fp32's exponents.
template <bool BF>
constexpr float kTopWeight = BF ? 0.f : 15.f;
constexpr int kRowTile = 16, kRowWarps = 4;
cudaError_t launch_paged_rows(const AttnParams& p, bool bf16, cudaStream_t st);
constexpr int kPairRows = 256;
cudaError_t launch_paged_chunk(const AttnParams& p, bool bf16, cudaStream_t st);
cudaError_t launch_paged_join(const AttnParams& p, bool bf16, cudaStream_t st);

// ---- pages (pages.cu)
cudaError_t launch_pages_fork(int32_t* refs, int P, int32_t* table, long long ts, int width,
                              int32_t* lens, int S, const int32_t* src, const int32_t* dst, int F,
                              int32_t* refused, cudaStream_t st);
cudaError_t launch_pages_reserve(int32_t* refs, int P, int32_t* table, long long ts, int width,
                                 int32_t* lens, const int32_t* add, int S, int page,
                                 int32_t* moves, int32_t* status, int32_t* scratch,
                                 cudaStream_t st);
cudaError_t launch_pages_free(int32_t* refs, int P, int32_t* table, long long ts, int width,
                              int32_t* lens, int S, const int32_t* slots, int F, cudaStream_t st);
cudaError_t launch_pages_compact(int32_t* refs, int P, int32_t* table, long long ts, int width,
                                 int S, int32_t* moves, int32_t* count, int32_t* scratch,
                                 cudaStream_t st);
cudaError_t launch_pages_copy(uint8_t* pools, int B, long long pool_stride, int P,
                              long long page_stride, long long page_bytes, const int32_t* moves,
                              int M, const int32_t* count, cudaStream_t st);

// device address of the error word (paged_api.cu)
int* paged_error_word();
// multiprocessors of the current device
int device_sms();
// Lets `kern` have `bytes` of dynamic shared memory on the current device, where it
// takes effect; `done`, the kernel's own, says on which it has been set.
cudaError_t allow_smem(const void* kern, int bytes, std::atomic<uint64_t>& done);

}  // namespace moe
