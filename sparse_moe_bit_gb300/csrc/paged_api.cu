// C ABI of the paged-cache operators (include/paged.h): argument checks, the
// choice of kernel and split, launches on the caller's stream.
#include <cmath>
#include <cstring>

#include "paged_internal.h"

using namespace moe;

namespace moe {

namespace {
__device__ int g_paged_err;
constexpr int kMaxDevices = 64;
__global__ void clear_bits_kernel(int* word, int bits) { atomicAnd(word, ~bits); }
}  // namespace

static cudaError_t launch_clear_bits(int* word, int bits, cudaStream_t st) {
  return launch_kernel(clear_bits_kernel, dim3(1), dim3(1), 0, st, word, bits);
}

int* paged_error_word() {
  static int* at[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  if (!at[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_paged_err) != cudaSuccess) return nullptr;
    at[dev] = static_cast<int*>(p);
  }
  return at[dev];
}

int device_sms() {
  static int sms[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 152;
  if (!sms[dev]) {
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v < 1)
      v = 152;
    sms[dev] = v;
  }
  return sms[dev];
}

cudaError_t allow_smem(const void* kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < kMaxDevices ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

bool make_page_map(CUtensorMap* m, const void* base, const CacheView& c, int features, int box,
                   bool bf16) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);
  static Encode encode = nullptr;
  if (!encode) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    encode = reinterpret_cast<Encode>(f);
  }
  const cuuint64_t dims[4] = {(cuuint64_t)c.dim, (cuuint64_t)c.page, (cuuint64_t)c.heads,
                              (cuuint64_t)c.pages};
  // (a dimension of one element is never stepped along: any stride will do)
  const cuuint64_t strides[3] = {c.page == 1 ? 16 : (cuuint64_t)c.row_stride * 2,
                                 c.heads == 1 ? 16 : (cuuint64_t)c.head_stride * 2,
                                 c.pages == 1 ? 16 : (cuuint64_t)c.page_stride * 2};
  const cuuint32_t boxes[4] = {(cuuint32_t)features, (cuuint32_t)box, 1, 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  return encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                const_cast<void*>(base), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                features == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

#define PAGED_CK(call, what)                                                             \
  do {                                                                                   \
    const cudaError_t e_ = (call);                                                       \
    if (e_ != cudaSuccess)                                                               \
      return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e_));                 \
  } while (0)

moe_status check_cache(const paged_cache* c, CacheView* v) {
  if (!c) return fail(MOE_ERR_INVALID_ARG, "cache is NULL");
  if (c->dtype != PAGED_BF16 && c->dtype != PAGED_F16)
    return fail(MOE_ERR_INVALID_ARG, "cache dtype %d", c->dtype);
  if (c->pages < 1 || c->page < 1 || c->heads < 1)
    return fail(MOE_ERR_INVALID_ARG, "bad cache (pages=%d page=%d heads=%d)", c->pages, c->page,
                c->heads);
  if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
    return fail(MOE_ERR_INVALID_ARG, "cache arrays NULL or not 16-byte aligned");
  if (c->page_stride < 0 || c->row_stride < 0 || c->head_stride < 0 || c->page_stride % 8 ||
      c->row_stride % 8 || c->head_stride % 8)
    return fail(MOE_ERR_INVALID_ARG, "cache strides must be multiples of 8 elements");
  if (c->dim != 64 && c->dim != 128 && c->dim != 256)
    return fail(MOE_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128, 256)", c->dim);
  v->k = static_cast<uint16_t*>(c->k);
  v->v = static_cast<uint16_t*>(c->v);
  v->pages = c->pages;
  v->page = c->page;
  v->heads = c->heads;
  v->dim = c->dim;
  v->page_stride = c->page_stride;
  v->row_stride = c->row_stride;
  v->head_stride = c->head_stride;
  v->div = make_fastdiv(c->page);
  return MOE_OK;
}

moe_status check_batch(const paged_batch* b, int page, BatchView* v) {
  if (!b) return fail(MOE_ERR_INVALID_ARG, "batch is NULL");
  if (b->N < 0 || b->T < 0 || b->width < 0 || b->table_stride < 0)
    return fail(MOE_ERR_INVALID_ARG, "bad batch (N=%d T=%d width=%d)", b->N, b->T, b->width);
  if (b->N > 0 && b->T > 0 && (!b->cu_q || !b->kv_len || (b->width > 0 && !b->table)))
    return fail(MOE_ERR_INVALID_ARG, "NULL batch array");
  if (!aligned(b->cu_q, 4) || !aligned(b->kv_len, 4) || !aligned(b->table, 4))
    return fail(MOE_ERR_INVALID_ARG, "misaligned batch array");
  v->table = b->table;
  v->cu = b->cu_q;
  v->kv_len = b->kv_len;
  v->N = b->N;
  v->T = b->T;
  v->width = b->width;
  v->table_stride = b->table_stride;
  const long long cap = (long long)b->width * page;
  v->capacity = cap > 0x7fffff00ll ? 0x7fffff00 : (int)cap;
  return MOE_OK;
}

moe_status check_rope(int D, const double* freq, int r, float mscale) {
  if (r < 1 || 2 * r > D || D > 1024)
    return fail(MOE_ERR_INVALID_ARG, "%d frequencies for heads of %d features", r, D);
  if (!freq || !aligned(freq, 8)) return fail(MOE_ERR_INVALID_ARG, "freq NULL or misaligned");
  if (!std::isfinite(mscale)) return fail(MOE_ERR_INVALID_ARG, "mscale is not finite");
  return MOE_OK;
}

// Choice of kernel and split for one attention over a batch.
struct Plan {
  bool wide;  // 256-row tiles on the tensor cores, else 8- or 16-row tiles
  int tiles, chunks, chunk;  // 256-row tiles
  int warps, row_tile;       // small tiles
  int parts;                 // of a row, about
  size_t ml, before, ws;     // offsets of the partial maxima and sums, of the counts; total bytes
};

// Tiles of 8 or 16 rows while one holds the longest chunk's rows (each tile reads
// the keys again), 256-row tiles above.  Where the caller does not say how long the
// longest chunk is, the mean stands for it, which is that length for a decode batch; of
// more tokens than sequences, which may lie in one chunk, up to half a tile: its tiles'
// reads then add at most half to those of the others.  Measured without max_q, small
// tiles and 256-row ones: 64 ragged contexts up to 8192 that decode 112 and 154 us (16/2
// heads of 256; 32/8 of 128: 200 and 257); 8/8 heads of 128, 63 of them and a chunk of
// 128 tokens, 3 rows in the mean, 217 and 257; 99 contexts of 4096 and a chunk of 1000,
// 11 rows, 387 and 353; 127 of 32768 and one of 1900, 16 rows, 4666 and 2903.
//
// Small tiles: as many warps as the SMs hold, four each (a warp's ring takes a
// quarter of the shared memory), but at least two groups of keys (16 KB each) for
// a warp.
// 256-row tiles: split over the keys only while the pairs of CTAs leave SMs
// without work; no chunk below 512 keys.
//
// The keys that a group shares may be read again for every 16 rows where that is little:
// 256-row tiles take some 10 us more than small ones before their first product (4
// continuations of 1501 keys, 16/2 heads of 256, 2 tiles of 16 rows: 25 us a call's
// kernels, 30 with 256-row tiles).  Their split over the keys goes by the tiles that are
// likely there (5 groups, 57 sequences, 24/8 heads of 128: 84 us, 92 without).
constexpr double kReread = 48 << 20;
Plan plan(const CacheView& c, const BatchView& b, int Hq, int window, int max_q, int max_kv,
          bool group = false) {
  Plan r{};
  const int G = Hq / c.heads;
  long long mq = max_q > 0 ? max_q : b.N > 0 ? ((long long)b.T + b.N - 1) / b.N : b.T;
  if (mq > b.T) mq = b.T;
  long long kv = max_kv > 0 ? max_kv : b.capacity;
  if (kv > b.capacity) kv = b.capacity;
  r.wide = mq * G > (max_q > 0 || b.T <= b.N ? kRowTile : kRowTile / 2);
  if (group && r.wide)
    r.wide = (double)((mq * G + kRowTile - 1) / kRowTile) * b.N * kv * c.heads * c.dim * 4 > kReread;
  r.row_tile = mq * G <= 8 ? 8 : kRowTile;
  const long long rows = r.wide ? kPairRows : r.row_tile;
  long long span = kv;
  if (window > 0 && window + rows < span) span = window + rows;
  r.tiles = r.chunks = r.chunk = 1;
  size_t parts;
  if (r.wide) {
    long long tiles = ((long long)b.T * G + rows - 1) / rows + (b.N < b.T ? b.N : b.T);
    if (b.N == 1) --tiles;
    if (tiles < 1) tiles = 1;
    const long long items = tiles * c.heads;
    long long chunks = device_sms() / 2 / items;
    if (group) {  // (of the tiles that each group may have beyond its rows half are there)
      const long long likely = (((long long)b.T * G + rows - 1) / rows + b.N / 2) * c.heads;
      chunks = (device_sms() / 2 + likely / 2) / likely;
    }
    if (chunks < 1) chunks = 1;
    long long chunk = (span + chunks - 1) / chunks;
    chunk = (chunk + 127) / 128 * 128;
    if (chunk < 512) chunk = 512;
    chunks = (span + chunk - 1) / chunk;
    if (chunks < 1) chunks = 1;
    r.tiles = (int)tiles;
    r.chunk = (int)chunk;
    r.chunks = (int)chunks;
    parts = r.chunks > 1 ? (size_t)b.T * Hq * r.chunks : 0;
    r.parts = r.chunks;
  } else {
    const long long tiles = (mq * G + rows - 1) / rows;
    const int kg = 4096 / c.dim;  // keys of a group
    const long long items = (long long)b.N * tiles * c.heads;
    const long long groups = items * ((span + kg - 1) / kg);
    const long long most = (long long)kRowWarps * device_sms();
    long long warps = groups / 2 / kRowWarps * kRowWarps;
    if (warps < kRowWarps) warps = kRowWarps;
    r.warps = (int)(warps < most ? warps : most);
    r.parts = (int)(r.warps / (items > 0 ? items : 1)) + 1;
    parts = (size_t)2 * r.warps * kRowTile;
  }
  r.ml = parts * c.dim * 4;
  r.before = (r.ml + parts * 8 + 255) / 256 * 256;
  r.ws = r.before + (r.wide ? 0 : ((size_t)b.N + 1) * 8);
  return r;
}

void set_plan(AttnParams* p, const Plan& r, void* workspace) {
  p->tiles = r.tiles;
  p->chunks = r.chunks;
  p->chunk = r.chunk;
  p->split = r.wide && r.chunks > 1;
  p->warps = r.warps;
  p->row_tile = r.row_tile;
  p->parts = r.parts;
  p->part_o = static_cast<float*>(workspace);
  p->part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + r.ml);
  p->before = reinterpret_cast<long long*>(static_cast<uint8_t*>(workspace) + r.before);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// An attention over shared keys: plans of the groups as a batch and of the sequences' own
// keys, whose results are partial, whatever their split; behind them the results that a
// warp of the small tiles has whole, and the groups.
struct SharedPlan {
  Plan g, p;
  // small tiles for both: one batch of the groups and the sequences, one launch (g is its
  // plan; 4 continuations of 1501 keys, 16/2 heads of 256: 29 us a call, 33 with a launch
  // for each; groups of 1, 2 and 3 sequences 29 and 66)
  bool one;
  int N;  // sequences of the batch that g is of
  size_t at_p, whole_g, whole_p, groups, ws;
};
SharedPlan plan_shared(const CacheView& c, const BatchView& b, int Hq, int G, int max_q, int max_group,
                       int max_shared, int max_tail) {
  SharedPlan r{};
  BatchView gb = b;
  gb.N = G;
  r.g = plan(c, gb, Hq, 0, max_group, max_shared, true);
  r.p = plan(c, b, Hq, 0, max_q, max_tail);
  const size_t rows = (size_t)b.T * Hq, row = (size_t)c.dim * 4 + 8;
  r.one = !r.g.wide && !r.p.wide && (long long)G + b.N < 0x7ffffff0;
  r.N = r.one ? G + 1 + b.N : G;
  if (r.one) {
    const int most = kRowWarps * device_sms();
    r.g.warps = r.g.warps + r.p.warps < most ? r.g.warps + r.p.warps : most;
    r.g.row_tile = r.g.row_tile > r.p.row_tile ? r.g.row_tile : r.p.row_tile;
    r.g.parts = (r.g.parts + r.p.parts + 1) / 2;
    r.g.ml = (size_t)2 * r.g.warps * kRowTile * c.dim * 4;
    r.g.before = up256(r.g.ml + (size_t)2 * r.g.warps * kRowTile * 8);
    r.whole_g = up256(r.g.before + ((size_t)r.N + 1) * 8);
    r.groups = r.whole_g + up256(2 * rows * row);
    r.ws = r.groups + (size_t)b.T * 8 + ((size_t)4 * r.N + 1) * 4;
    return r;
  }
  for (Plan* x : {&r.g, &r.p}) {
    if (!x->wide || x->chunks > 1) continue;
    x->ml = rows * c.dim * 4;
    x->before = x->ws = up256(x->ml + rows * 8);
  }
  r.at_p = up256(r.g.ws);
  r.whole_g = r.at_p + up256(r.p.ws);
  r.whole_p = r.whole_g + (r.g.wide ? 0 : up256(rows * row));
  r.groups = r.whole_p + (r.p.wide ? 0 : up256(rows * row));
  r.ws = r.groups + (size_t)b.T * 8 + ((size_t)3 * G + 1 + b.N) * 4;
  return r;
}

moe_status check_attention(const paged_cache* cache, const paged_batch* batch, int Hq, int window,
                           int max_q, int max_kv, CacheView* c, BatchView* b) {
  moe_status s = check_cache(cache, c);
  if (s != MOE_OK) return s;
  s = check_batch(batch, cache->page, b);
  if (s != MOE_OK) return s;
  if (Hq < 1 || Hq % cache->heads)
    return fail(MOE_ERR_INVALID_ARG, "%d query heads on %d key/value heads", Hq, cache->heads);
  if (window < 0 || max_q < 0 || max_kv < 0)
    return fail(MOE_ERR_INVALID_ARG, "negative window, max_q or max_kv");
  if ((long long)batch->T * Hq >= (1ll << 31) - 256)
    return fail(MOE_ERR_UNSUPPORTED, "T * Hq = %lld", (long long)batch->T * Hq);
  return MOE_OK;
}

// An attention call's arguments; p gets all of them but the mask and the split.
moe_status check_queries(const void* q, int64_t q_ts, int64_t q_hs, int Hq, const paged_cache* cache,
                         const paged_batch* batch, float scale, int window, int max_q, int max_kv,
                         void* o, int64_t o_ts, int64_t o_hs, float* lse, void* workspace,
                         AttnParams* p) {
  moe_status s = check_attention(cache, batch, Hq, window, max_q, max_kv, &p->c, &p->b);
  if (s != MOE_OK) return s;
  if (!(scale > 0) || !std::isfinite(scale))
    return fail(MOE_ERR_INVALID_ARG, "scale must be positive and finite");
  if (batch->T == 0 || batch->N == 0) return MOE_OK;
  if (!q || !o) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 16))
    return fail(MOE_ERR_INVALID_ARG, "misaligned pointer");
  if (q_ts % 8 || q_hs % 8 || o_ts % 8 || o_hs % 8 || q_ts < 0 || q_hs < 0 || o_ts < 0 || o_hs < 0)
    return fail(MOE_ERR_INVALID_ARG, "strides must be multiples of 8 elements");
  p->q = static_cast<const uint16_t*>(q);
  p->o = static_cast<uint16_t*>(o);
  p->lse = lse;
  p->q_ts = q_ts;
  p->q_hs = q_hs;
  p->o_ts = o_ts;
  p->o_hs = o_hs;
  p->Hq = Hq;
  p->G = Hq / cache->heads;
  p->divG = make_fastdiv(p->G);
  p->scale_log2 = scale * 1.44269504088896340736f;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status rope_frequencies(int rot, double base, int scaling, double factor, double original,
                            double low, double high, double* freq, double* mscale) {
  if (rot < 2 || rot % 2) return fail(MOE_ERR_INVALID_ARG, "rot=%d", rot);
  if (!freq || !mscale) return fail(MOE_ERR_INVALID_ARG, "NULL output");
  if (!(base > 0) || !std::isfinite(base)) return fail(MOE_ERR_INVALID_ARG, "base must be positive");
  if (scaling < ROPE_SCALE_NONE || scaling > ROPE_SCALE_BANDED)
    return fail(MOE_ERR_INVALID_ARG, "scaling %d", scaling);
  if (scaling != ROPE_SCALE_NONE && (!(factor > 0) || !std::isfinite(factor)))
    return fail(MOE_ERR_INVALID_ARG, "factor must be positive");
  if (scaling == ROPE_SCALE_NTK && rot < 4)
    return fail(MOE_ERR_INVALID_ARG, "this scaling needs rot > 2");
  const bool band = scaling == ROPE_SCALE_YARN || scaling == ROPE_SCALE_BANDED;
  if (band && (!(original > 0) || !(low > 0) || !(high > low) || !std::isfinite(original) ||
               !std::isfinite(high)))
    return fail(MOE_ERR_INVALID_ARG, "original, low and high must be positive with low < high");
  if (scaling == ROPE_SCALE_YARN && base == 1.0)
    return fail(MOE_ERR_INVALID_ARG, "base 1 has no ramp");
  const double two_pi = 6.283185307179586476925;
  const int r = rot / 2;
  *mscale = 1.0;
  if (scaling == ROPE_SCALE_NTK) base *= std::pow(factor, (double)rot / (rot - 2));
  // the (fractional) pair that turns `t` times within `original` positions
  auto pair_of = [&](double t) {
    return rot * std::log(original / (t * two_pi)) / (2 * std::log(base));
  };
  double lo = 0, hi = 1;
  if (scaling == ROPE_SCALE_YARN) {
    lo = std::fmax(std::floor(pair_of(high)), 0.0);
    hi = std::fmin(std::ceil(pair_of(low)), (double)rot - 1);
    if (hi - lo < 1e-3) hi = lo + 1e-3;
    if (factor > 1) *mscale = 0.1 * std::log(factor) + 1.0;
  }
  for (int i = 0; i < r; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == ROPE_SCALE_LINEAR) f /= factor;
    if (scaling == ROPE_SCALE_YARN) {
      const double ramp = std::fmin(std::fmax((i - lo) / (hi - lo), 0.0), 1.0);
      f = f / factor * ramp + f * (1 - ramp);
    }
    if (scaling == ROPE_SCALE_BANDED) {
      const double turns = original * f / two_pi;
      const double s = std::fmin(std::fmax((turns - low) / (high - low), 0.0), 1.0);
      f = f * (s + (1 - s) / factor);
    }
    freq[i] = f;
  }
  return MOE_OK;
}

moe_status rope(const void* x, void* out, int dtype, int T, int H, int D, int64_t x_ts,
                int64_t x_hs, int64_t o_ts, int64_t o_hs, const int32_t* pos, const double* freq,
                int r, float mscale, int interleaved, int inverse, void* stream) {
  if (dtype != PAGED_BF16 && dtype != PAGED_F16 && dtype != PAGED_F32)
    return fail(MOE_ERR_INVALID_ARG, "dtype %d", dtype);
  if (T < 0 || H < 1 || D < 1) return fail(MOE_ERR_INVALID_ARG, "bad size (T=%d H=%d D=%d)", T, H, D);
  moe_status s = check_rope(D, freq, r, mscale);
  if (s != MOE_OK) return s;
  if (T == 0) return MOE_OK;
  if (!x || !out || !pos) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  const size_t es = dtype == PAGED_F32 ? 4 : 2;
  if (!aligned(x, es) || !aligned(out, es) || !aligned(pos, 4))
    return fail(MOE_ERR_INVALID_ARG, "misaligned pointer");
  if (x == out && (x_ts != o_ts || x_hs != o_hs))
    return fail(MOE_ERR_INVALID_ARG, "in place with other strides");
  if ((long long)H * D > (1 << 24)) return fail(MOE_ERR_UNSUPPORTED, "H * D above 2^24");
  RopeParams p{};
  p.x = x;
  p.out = out;
  p.T = T;
  p.H = H;
  p.D = D;
  p.x_ts = x_ts;
  p.x_hs = x_hs;
  p.o_ts = o_ts;
  p.o_hs = o_hs;
  p.pos = pos;
  p.freq = freq;
  p.r = r;
  p.mscale = mscale;
  p.sign = inverse ? -1.f : 1.f;
  p.interleaved = interleaved != 0;
  p.in_place = x == out;
  PAGED_CK(launch_rope(p, dtype, false, static_cast<cudaStream_t>(stream)), "rope launch");
  return MOE_OK;
}

moe_status rope_append(const void* q, int64_t q_ts, void* q_out, int Hq, const void* k,
                       int64_t k_ts, const void* v, int64_t v_ts, const paged_cache* cache,
                       const paged_batch* batch, const double* freq, int r, float mscale,
                       int interleaved, void* stream) {
  RopeParams p{};
  moe_status s = check_cache(cache, &p.c);
  if (s != MOE_OK) return s;
  s = check_batch(batch, cache->page, &p.b);
  if (s != MOE_OK) return s;
  if (Hq < 1) return fail(MOE_ERR_INVALID_ARG, "Hq=%d", Hq);
  s = check_rope(cache->dim, freq, r, mscale);
  if (s != MOE_OK) return s;
  if (batch->T == 0 || batch->N == 0) return MOE_OK;
  if (!q || !q_out || !k || !v) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  if (!aligned(q, 2) || !aligned(q_out, 2) || !aligned(k, 2) || !aligned(v, 2))
    return fail(MOE_ERR_INVALID_ARG, "misaligned pointer");
  if ((long long)(Hq + 2 * cache->heads) * cache->dim > (1 << 24))
    return fail(MOE_ERR_UNSUPPORTED, "heads * dim above 2^24");
  const long long D = cache->dim;
  if (q == q_out && q_ts != Hq * D)
    return fail(MOE_ERR_INVALID_ARG, "q in place must be dense");
  p.x = q;
  p.out = q_out;
  p.T = batch->T;
  p.H = Hq;
  p.D = (int)D;
  p.x_ts = q_ts;
  p.x_hs = D;
  p.o_ts = Hq * D;
  p.o_hs = D;
  p.freq = freq;
  p.r = r;
  p.mscale = mscale;
  p.sign = 1.f;
  p.interleaved = interleaved != 0;
  p.in_place = q == q_out;
  p.k = k;
  p.v = v;
  p.k_ts = k_ts;
  p.v_ts = v_ts;
  p.err = paged_error_word();
  if (!p.err) return fail(MOE_ERR_CUDA, "no CUDA device");
  PAGED_CK(launch_rope(p, cache->dtype, true, static_cast<cudaStream_t>(stream)),
           "rope_append launch");
  return MOE_OK;
}

moe_status paged_attention_workspace(const paged_cache* cache, const paged_batch* batch, int Hq,
                                     int window, int max_q, int max_kv, size_t* bytes) {
  if (!bytes) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  CacheView c;
  BatchView b;
  moe_status s = check_attention(cache, batch, Hq, window, max_q, max_kv, &c, &b);
  if (s != MOE_OK) return s;
  *bytes = plan(c, b, Hq, window, max_q, max_kv).ws;
  return MOE_OK;
}

moe_status paged_attention(const void* q, int64_t q_ts, int64_t q_hs, int Hq,
                           const paged_cache* cache, const paged_batch* batch, float scale,
                           int causal, int window, int max_q, int max_kv, void* o, int64_t o_ts,
                           int64_t o_hs, float* lse, void* workspace, size_t workspace_bytes,
                           void* stream) {
  AttnParams p{};
  moe_status s = check_queries(q, q_ts, q_hs, Hq, cache, batch, scale, window, max_q, max_kv, o, o_ts,
                               o_hs, lse, workspace, &p);
  if (s != MOE_OK || batch->T == 0 || batch->N == 0) return s;
  const Plan r = plan(p.c, p.b, Hq, window, max_q, max_kv);
  if (r.ws > 0 && (!workspace || workspace_bytes < r.ws))
    return fail(MOE_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, r.ws);
  if (2ll * r.tiles * p.c.heads * r.chunks >= (1ll << 31))
    return fail(MOE_ERR_UNSUPPORTED, "too many row tiles");
  p.err = paged_error_word();
  if (!p.err) return fail(MOE_ERR_CUDA, "no CUDA device");
  p.causal = causal != 0;
  p.window = window;
  set_plan(&p, r, workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = cache->dtype == PAGED_BF16;
  PAGED_CK(r.wide ? launch_paged_chunk(p, bf, st) : launch_paged_rows(p, bf, st),
           "paged_attention launch");
  if (!r.wide || r.chunks > 1) PAGED_CK(launch_paged_join(p, bf, st), "paged_attention join launch");
  return MOE_OK;
}

moe_status paged_attention_shared_workspace(const paged_cache* cache, const paged_batch* batch,
                                            int Hq, int groups, int max_q, int max_group,
                                            int max_shared, int max_tail, size_t* bytes) {
  if (!bytes) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  CacheView c;
  BatchView b{};
  moe_status s = check_attention(cache, batch, Hq, 0, max_q, max_tail, &c, &b);
  if (s != MOE_OK) return s;
  if (groups < 0 || max_group < 0 || max_shared < 0)
    return fail(MOE_ERR_INVALID_ARG, "negative groups, max_group or max_shared");
  *bytes = groups == 0 ? plan(c, b, Hq, 0, max_q, max_tail).ws
                       : plan_shared(c, b, Hq, groups, max_q, max_group, max_shared, max_tail).ws;
  return MOE_OK;
}

moe_status paged_attention_shared(const void* q, int64_t q_ts, int64_t q_hs, int Hq,
                                  const paged_cache* cache, const paged_batch* batch,
                                  const int32_t* cu_group, const int32_t* shared, int groups,
                                  float scale, int causal, int max_q, int max_group, int max_shared,
                                  int max_tail, void* o, int64_t o_ts, int64_t o_hs, float* lse,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  if (groups < 0 || max_group < 0 || max_shared < 0)
    return fail(MOE_ERR_INVALID_ARG, "negative groups, max_group or max_shared");
  if (groups == 0)
    return paged_attention(q, q_ts, q_hs, Hq, cache, batch, scale, causal, 0, max_q, max_tail, o, o_ts,
                           o_hs, lse, workspace, workspace_bytes, stream);
  AttnParams p{};
  moe_status s = check_queries(q, q_ts, q_hs, Hq, cache, batch, scale, 0, max_q, max_tail, o, o_ts, o_hs,
                               lse, workspace, &p);
  if (s != MOE_OK || batch->T == 0 || batch->N == 0) return s;
  if (!cu_group || !shared || !aligned(cu_group, 4) || !aligned(shared, 4))
    return fail(MOE_ERR_INVALID_ARG, "cu_group or shared NULL or misaligned");
  const SharedPlan r = plan_shared(p.c, p.b, Hq, groups, max_q, max_group, max_shared, max_tail);
  if (!workspace || workspace_bytes < r.ws)
    return fail(MOE_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, r.ws);
  for (const Plan* x : {&r.g, &r.p})
    if (2ll * x->tiles * p.c.heads * x->chunks >= (1ll << 31))
      return fail(MOE_ERR_UNSUPPORTED, "too many row tiles");
  p.err = paged_error_word();
  if (!p.err) return fail(MOE_ERR_CUDA, "no CUDA device");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t rows = (size_t)p.b.T * Hq, whole_ml = rows * p.c.dim * 4;
  GroupView gv{};
  gv.cu_group = cu_group;
  gv.shared = shared;
  gv.G = groups;
  gv.of_token = reinterpret_cast<int2*>(ws + r.groups);
  gv.cu = reinterpret_cast<int32_t*>(ws + r.groups + (size_t)p.b.T * 8);
  gv.len = gv.cu + r.N + 1;
  gv.rows = gv.len + r.N;
  gv.skip = gv.rows + r.N;
  gv.own = r.one ? groups + 1 : 0;
  AttnParams g = p;
  set_plan(&g, r.g, ws);
  g.split = r.g.wide;
  g.causal = r.one && causal;
  g.flat = groups;
  g.early = 1;
  g.b.N = r.N;
  g.b.cu = gv.cu;
  g.b.kv_len = gv.len;
  g.b.rows = gv.rows;
  if (!r.g.wide) {
    g.whole_o = reinterpret_cast<float*>(ws + r.whole_g);
    g.whole_ml = reinterpret_cast<float2*>(ws + r.whole_g + (r.one ? 2 : 1) * whole_ml);
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = cache->dtype == PAGED_BF16;
  PAGED_CK(launch_paged_groups(p.b, gv, st), "paged_attention_shared groups launch");
  if (r.one) {
    g.flat_rows = (long long)rows;
    g.b.skip = gv.skip;
    PAGED_CK(launch_paged_rows(g, bf, st), "paged_attention_shared launch");
    PAGED_CK(launch_paged_join_shared(g, g, gv.of_token, gv.own, bf, st), "paged_attention_shared join launch");
    return MOE_OK;
  }
  set_plan(&p, r.p, ws + r.at_p);
  p.causal = causal != 0;
  p.split = r.p.wide;
  if (!r.p.wide) {
    p.whole_o = reinterpret_cast<float*>(ws + r.whole_p);
    p.whole_ml = reinterpret_cast<float2*>(ws + r.whole_p + whole_ml);
  }
  p.b.skip = gv.skip;
  p.late = 1;
  PAGED_CK(r.g.wide ? launch_paged_chunk(g, bf, st) : launch_paged_rows(g, bf, st),
           "paged_attention_shared launch");
  PAGED_CK(r.p.wide ? launch_paged_chunk(p, bf, st) : launch_paged_rows(p, bf, st),
           "paged_attention_shared launch");
  PAGED_CK(launch_paged_join_shared(p, g, gv.of_token, 0, bf, st), "paged_attention_shared join launch");
  return MOE_OK;
}

static moe_status check_pages(const int32_t* refs, int P, const int32_t* table, int64_t ts,
                              int width, const int32_t* lens, int S) {
  if (P < 1 || S < 0 || width < 0 || ts < 0)
    return fail(MOE_ERR_INVALID_ARG, "bad size (P=%d S=%d width=%d)", P, S, width);
  if ((long long)S * width >= (1ll << 31) || P > (1 << 30))
    return fail(MOE_ERR_UNSUPPORTED, "S * width = %lld, P = %d", (long long)S * width, P);
  if (!refs || (S > 0 && (!lens || (width > 0 && !table))))
    return fail(MOE_ERR_INVALID_ARG, "NULL state array");
  if (!aligned(refs, 4) || !aligned(table, 4) || !aligned(lens, 4))
    return fail(MOE_ERR_INVALID_ARG, "misaligned state array");
  if (S > 1 && ts < width) return fail(MOE_ERR_INVALID_ARG, "rows of the table overlap");
  return MOE_OK;
}

moe_status pages_fork(int32_t* refs, int P, int32_t* table, int64_t ts, int width, int32_t* lens,
                      int S, const int32_t* src, const int32_t* dst, int F, int32_t* refused,
                      void* stream) {
  moe_status s = check_pages(refs, P, table, ts, width, lens, S);
  if (s != MOE_OK) return s;
  if (F < 0) return fail(MOE_ERR_INVALID_ARG, "F=%d", F);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!aligned(refused, 4)) return fail(MOE_ERR_INVALID_ARG, "misaligned pointer");
  if (F > 0 && (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)))
    return fail(MOE_ERR_INVALID_ARG, "src or dst NULL or misaligned");
  if (refused) PAGED_CK(cudaMemsetAsync(refused, 0, 4, st), "clear");
  if (F == 0) return MOE_OK;
  PAGED_CK(launch_pages_fork(refs, P, table, ts, width, lens, S, src, dst, F, refused, st),
           "pages_fork launch");
  return MOE_OK;
}

moe_status pages_reserve(int32_t* refs, int P, int32_t* table, int64_t ts, int width,
                         int32_t* lens, const int32_t* add, int S, int page, int32_t* moves,
                         int32_t* status, int32_t* scratch, void* stream) {
  moe_status s = check_pages(refs, P, table, ts, width, lens, S);
  if (s != MOE_OK) return s;
  if (page < 1) return fail(MOE_ERR_INVALID_ARG, "page=%d", page);
  if (!status || !scratch || (S > 0 && (!add || !moves)))
    return fail(MOE_ERR_INVALID_ARG, "NULL array");
  if (!aligned(add, 4) || !aligned(moves, 4) || !aligned(status, 4) || !aligned(scratch, 4))
    return fail(MOE_ERR_INVALID_ARG, "misaligned array");
  PAGED_CK(launch_pages_reserve(refs, P, table, ts, width, lens, add, S, page, moves, status,
                                scratch, static_cast<cudaStream_t>(stream)),
           "pages_reserve launch");
  return MOE_OK;
}

moe_status pages_free(int32_t* refs, int P, int32_t* table, int64_t ts, int width, int32_t* lens,
                      int S, const int32_t* slots, int F, void* stream) {
  moe_status s = check_pages(refs, P, table, ts, width, lens, S);
  if (s != MOE_OK) return s;
  if (F < 0) return fail(MOE_ERR_INVALID_ARG, "F=%d", F);
  if (F == 0) return MOE_OK;
  if (!slots || !aligned(slots, 4)) return fail(MOE_ERR_INVALID_ARG, "slots NULL or misaligned");
  PAGED_CK(launch_pages_free(refs, P, table, ts, width, lens, S, slots, F,
                             static_cast<cudaStream_t>(stream)),
           "pages_free launch");
  return MOE_OK;
}

moe_status pages_compact(int32_t* refs, int P, int32_t* table, int64_t ts, int width, int S,
                         int32_t* moves, int32_t* count, int32_t* scratch, void* stream) {
  moe_status s = check_pages(refs, P, table, ts, width, refs, S);
  if (s != MOE_OK) return s;
  if (!moves || !count || !scratch) return fail(MOE_ERR_INVALID_ARG, "NULL array");
  if (!aligned(moves, 4) || !aligned(count, 4) || !aligned(scratch, 4))
    return fail(MOE_ERR_INVALID_ARG, "misaligned array");
  PAGED_CK(launch_pages_compact(refs, P, table, ts, width, S, moves, count, scratch,
                                static_cast<cudaStream_t>(stream)),
           "pages_compact launch");
  return MOE_OK;
}

moe_status pages_copy(void* pools, int B, int64_t pool_stride, int P, int64_t page_stride,
                      int64_t page_bytes, const int32_t* moves, int M, const int32_t* count,
                      void* stream) {
  if (B < 0 || P < 1 || M < 0 || page_bytes < 0 || pool_stride < 0 || page_stride < 0)
    return fail(MOE_ERR_INVALID_ARG, "bad size (B=%d P=%d M=%d)", B, P, M);
  if (page_bytes % 16 || pool_stride % 16 || page_stride % 16 || !aligned(pools, 16))
    return fail(MOE_ERR_INVALID_ARG, "pools, strides and page bytes must be multiples of 16 bytes");
  if (P > 1 && page_stride < page_bytes) return fail(MOE_ERR_INVALID_ARG, "pages overlap");
  if (page_bytes > (1ll << 32)) return fail(MOE_ERR_UNSUPPORTED, "page of %lld bytes", (long long)page_bytes);
  if (B == 0 || M == 0 || page_bytes == 0) return MOE_OK;
  if (!pools || !moves || !aligned(moves, 4) || !aligned(count, 4))
    return fail(MOE_ERR_INVALID_ARG, "NULL or misaligned pointer");
  PAGED_CK(launch_pages_copy(static_cast<uint8_t*>(pools), B, pool_stride, P, page_stride,
                             page_bytes, moves, M, count, static_cast<cudaStream_t>(stream)),
           "pages_copy launch");
  return MOE_OK;
}

moe_status paged_get_device_error(void* stream, int* code) {
  if (!code) return fail(MOE_ERR_INVALID_ARG, "code is NULL");
  int* w = paged_error_word();
  if (!w) return fail(MOE_ERR_CUDA, "no CUDA device");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int v = 0;
  PAGED_CK(cudaMemcpyAsync(&v, w, 4, cudaMemcpyDeviceToHost, st), "read error word");
  PAGED_CK(cudaStreamSynchronize(st), "synchronise");
  if (v) {  // what was read and no more: kernels of other streams may set bits meanwhile
    PAGED_CK(launch_clear_bits(w, v, st), "clear error word");
    PAGED_CK(cudaStreamSynchronize(st), "synchronise");
  }
  *code = v;
  return v ? MOE_ERR_DEVICE : MOE_OK;
}

}  // extern "C"
