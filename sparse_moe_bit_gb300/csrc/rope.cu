// Rotary positions, alone and with the write of new keys and values into the
// paged cache (include/paged.h).
//
// Pair i of a head at position pos turns by theta = pos f_i.  Only theta modulo
// one turn matters, and that is exact in integers: with F = the 64-bit fraction of
// f_i / (2 pi) turns, the low 64 bits of pos * F are the fraction of a turn
// reached, off by at most pos 2^-64 -- where pos * f in fp32 is off by 0.03 rad at
// 2^20 positions.  Its top 32 bits, as a signed number of half turns, go to
// sincospif.  F comes from the bits of the fp64 frequency by integer products (the
// few fp64 units would serialise the CTAs).
//
// Bound: HBM, one read and one write of every value.  A CTA takes a few tokens,
// computes the r angles of each once into shared memory (they serve every head)
// and then moves 16 bytes of each side of a pair (eight pairs) a thread and step.
// (A thread that keeps its piece of the head, with its angles in registers, and
// walks the heads needs four times the registers and was slower by a factor of 1.1
// to 4: what counts is the loads that many threads have in flight.)
// Measured: 16385 tokens x 32 heads x 128, bf16, all turned: 46 us, 5.8 TB/s of
// reads and writes (0.87 of the copy rate, 40 registers); 8313 new tokens of 32
// query and 8 key/value heads of 128 into the cache 39.5 us, 0.77 of it.
// Vectors need r and the rest of the head (D - 2r) to be multiples of the 16 bytes' 8
// (fp32: 4) values, in either layout, and aligned rows; everything else takes the same
// loop one pair at a time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_internal.h"

namespace moe {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeCtas = 6;  // about so many CTAs an SM

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
  const float x = a * cs.x - b * cs.y;
  const float y = a * cs.y + b * cs.x;
  a = x;
  b = y;
}

// One head row: features of `src` turned into `dst`; item u of the row's
// items, V pairs (turning part) or V features (the rest) each.
template <typename T, int V, bool INTER>
__device__ __forceinline__ void rope_item(const T* src, T* dst, int u, int r, const float2* cs) {
  using W = Vec<T, V>;
  const int turns = r / V;  // items of V pairs
  if (u < turns) {
    if (INTER) {
      // V pairs = 2V consecutive features, as two vectors
      W x0 = reinterpret_cast<const W*>(src)[2 * u], x1 = reinterpret_cast<const W*>(src)[2 * u + 1];
      T t[2 * V];
#pragma unroll
      for (int j = 0; j < V; ++j) t[j] = x0.e[j], t[V + j] = x1.e[j];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float a = to_f(t[2 * j]), b = to_f(t[2 * j + 1]);
        turn(a, b, cs[j * turns + u]);
        t[2 * j] = from_f<T>(a);
        t[2 * j + 1] = from_f<T>(b);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) x0.e[j] = t[j], x1.e[j] = t[V + j];
      reinterpret_cast<W*>(dst)[2 * u] = x0;
      reinterpret_cast<W*>(dst)[2 * u + 1] = x1;
    } else {
      W a = reinterpret_cast<const W*>(src)[u], b = reinterpret_cast<const W*>(src + r)[u];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float fa = to_f(a.e[j]), fb = to_f(b.e[j]);
        turn(fa, fb, cs[j * turns + u]);
        a.e[j] = from_f<T>(fa);
        b.e[j] = from_f<T>(fb);
      }
      reinterpret_cast<W*>(dst)[u] = a;
      reinterpret_cast<W*>(dst + r)[u] = b;
    }
  } else {
    const int i = (2 * r) / V + (u - turns);
    reinterpret_cast<W*>(dst)[i] = reinterpret_cast<const W*>(src)[i];
  }
}

// The 64-bit fraction of freq / (2 pi) turns, freq's bits given.
__device__ __forceinline__ uint64_t turns_of(uint64_t bits) {
  const int ex = (int)(bits >> 52 & 2047);
  uint64_t man = bits & 0xfffffffffffffull;
  if (ex) man |= 1ull << 52;
  // freq = man 2^(e - 52); 1 / (2 pi) = kInv 2^-66; so turns 2^64 = man kInv 2^(e - 54)
  constexpr uint64_t kInv = 0xa2f9836e4e44152aull;
  const uint64_t hi = __umul64hi(man, kInv), lo = man * kInv;
  const int sh = 54 - ((ex ? ex : 1) - 1023);  // to the right
  uint64_t f = 0;
  if (sh >= 64)
    f = sh < 128 ? hi >> (sh - 64) : 0;
  else if (sh > 0)
    f = hi << (64 - sh) | lo >> sh;
  else
    f = sh > -64 ? lo << -sh : 0;
  return bits >> 63 ? 0 - f : f;
}

struct Slot {
  int pos;
  int seq;         // append: -1 = outside every sequence
  long long off;   // append: element offset of the token's row in k and v, -1 = none
};

template <typename T, int V, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  extern __shared__ float2 cs_all[];  // [tokens][r]
  __shared__ Slot slots[32];
  const int t0 = blockIdx.x * p.tokens;
  const int nt = min(p.tokens, p.T - t0);
  if (threadIdx.x < nt) {
    Slot s;
    const int t = t0 + threadIdx.x;
    if (APPEND) {
      s.off = -1;
      s.pos = 0;
      s.seq = find_seq(p.b, t);
      if (s.seq >= 0) {
        const Seq q = load_seq(p.b, s.seq);
        if (t >= q.t0 && t < q.t0 + q.nq) {
          // (kv_len as it is: clamped to the row's capacity it would put tokens that
          // have no place over the last ones that have)
          s.pos = max(p.b.kv_len[s.seq], 0) - q.nq + (t - q.t0);
          if (s.pos >= p.b.capacity) {
            atomicOr(p.err, PAGED_DEVERR_LENGTH);
          } else if (s.pos >= 0) {
            const int col = fast_div(s.pos, p.c.div);
            const int pg = p.b.table[s.seq * p.b.table_stride + col];
            if (pg >= 0 && pg < p.c.pages)
              s.off = pg * p.c.page_stride + (s.pos - col * p.c.page) * p.c.row_stride;
            else
              atomicOr(p.err, PAGED_DEVERR_PAGE);
          }
        } else {
          s.seq = -1;
        }
      }
    } else {
      s.seq = 0;
      s.off = -1;
      s.pos = p.pos[t];
    }
    slots[threadIdx.x] = s;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nt * p.r; i += kRopeThreads) {
    const int j = fast_div(i, p.div_r);
    const uint64_t bits = reinterpret_cast<const uint64_t*>(p.freq)[i - j * p.r];
    const uint64_t at = (uint64_t)(int64_t)slots[j].pos * turns_of(bits);  // modulo one turn
    const float half = (float)(int32_t)(at >> 32) * 4.656612873077393e-10f;  // 2^-31
    // (no angle where the frequency is not a number)
    const float scale = (bits >> 52 & 2047) == 2047 ? __int_as_float(0x7fffffff) : p.mscale;
    float s, c;
    sincospif(half, &s, &c);
    // (the V angles of a piece apart: pieces of neighbouring threads side by side)
    const int k = i - j * p.r;
    cs_all[j * p.r + k % V * (p.r / V) + k / V] = make_float2(c * scale, s * scale * p.sign);
  }
  __syncthreads();
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);
  const int rot_items = p.r / V;
  const int all_items = rot_items + (p.D - 2 * p.r) / V;
  const int q_items = (p.in_place ? rot_items : all_items);  // of a query row
  const int v_items = APPEND ? p.D / V : 0;
  const int heads = APPEND ? p.c.heads : 0;
  const int per_q = p.H * q_items, per_k = heads * all_items, per_v = heads * v_items;
  const int per_tok = per_q + per_k + per_v;
  for (int w = threadIdx.x; w < nt * per_tok; w += kRopeThreads) {
    const int j = fast_div(w, p.div_tok);
    int u = w - j * per_tok;
    const Slot s = slots[j];
    const long long t = t0 + j;
    const float2* cs = cs_all + j * p.r;
    if (APPEND && s.seq < 0) continue;
    if (u < per_q) {
      const int h = fast_div(u, p.div_q);
      rope_item<T, V, INTER>(x + t * p.x_ts + h * p.x_hs, out + t * p.o_ts + h * p.o_hs,
                             u - h * q_items, p.r, cs);
    } else if constexpr (APPEND) {
      if (s.off < 0) continue;
      u -= per_q;
      if (u < per_k) {
        const int h = fast_div(u, p.div_k);
        rope_item<T, V, INTER>(static_cast<const T*>(p.k) + t * p.k_ts + (long long)h * p.D,
                               reinterpret_cast<T*>(p.c.k) + s.off + h * p.c.head_stride,
                               u - h * all_items, p.r, cs);
      } else {
        u -= per_k;
        const int h = fast_div(u, p.div_v), i = u - h * v_items;
        using W = Vec<T, V>;
        const T* src = static_cast<const T*>(p.v) + t * p.v_ts + (long long)h * p.D;
        T* dst = reinterpret_cast<T*>(p.c.v) + s.off + h * p.c.head_stride;
        reinterpret_cast<W*>(dst)[i] = reinterpret_cast<const W*>(src)[i];
      }
    }
  }
}

template <typename T, int V>
cudaError_t launch_t(const RopeParams& p0, bool append, cudaStream_t st) {
  RopeParams p = p0;
  const int rot = p.r / V, all = rot + (p.D - 2 * p.r) / V, per_q = p.in_place ? rot : all;
  p.div_r = make_fastdiv(p.r);
  p.div_q = make_fastdiv(per_q);
  p.div_k = make_fastdiv(all);
  p.div_v = make_fastdiv(p.D / V > 0 ? p.D / V : 1);
  p.div_tok = make_fastdiv(p.H * per_q + (append ? p.c.heads * (all + p.D / V) : 0));
  // tokens of a CTA: one while the CTAs do not fill the machine three times over
  // (a small call is over in one token's time, and the last wave of a large one is
  // a small part), then up to eight, so that the lookups and angles of several
  // tokens take one round of latency
  const int full = device_sms() * kRopeCtas * 3;
  p.tokens = p.T / full;
  p.tokens = p.tokens < 1 ? 1 : (p.tokens > 8 ? 8 : p.tokens);
  const int grid = (p.T + p.tokens - 1) / p.tokens;
  const size_t smem = (size_t)p.tokens * p.r * sizeof(float2);
  void (*k)(RopeParams);
  if constexpr (sizeof(T) == 2)
    k = p.interleaved ? (append ? rope_kernel<T, V, true, true> : rope_kernel<T, V, true, false>)
                      : (append ? rope_kernel<T, V, false, true> : rope_kernel<T, V, false, false>);
  else
    k = p.interleaved ? rope_kernel<T, V, true, false> : rope_kernel<T, V, false, false>;
  return launch_kernel(k, dim3(grid), dim3(kRopeThreads), smem, st, p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, bool append, cudaStream_t st) {
  const int es = dtype == PAGED_F32 ? 4 : 2;
  const int V = 16 / es;
  // 16-byte vectors: whole vectors in each of the row's parts, aligned rows
  auto al = [&](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  bool vec = p.r % V == 0 && (p.D - 2 * p.r) % V == 0 && al(p.x) && al(p.out) && p.x_ts % V == 0 &&
             p.x_hs % V == 0 && p.o_ts % V == 0 && p.o_hs % V == 0;
  if (append) vec = vec && al(p.k) && al(p.v) && p.k_ts % V == 0 && p.v_ts % V == 0;
  if (dtype == PAGED_F32)
    return vec ? launch_t<float, 4>(p, false, st) : launch_t<float, 1>(p, false, st);
  if (dtype == PAGED_BF16)
    return vec ? launch_t<__nv_bfloat16, 8>(p, append, st)
               : launch_t<__nv_bfloat16, 1>(p, append, st);
  return vec ? launch_t<__half, 8>(p, append, st) : launch_t<__half, 1>(p, append, st);
}

}  // namespace moe
