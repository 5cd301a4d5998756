/*
 * sparse-moe-4bit for GB300 (sm_103a): C ABI of the attention layers' side of
 * the model, exported by the same library as moe.h (libmoe.so): rotary
 * positions, the write of new keys and values into a paged cache, attention
 * of new tokens over that cache, and the maintenance of its pages.
 *
 * Conventions are those of moe.h: device pointers, caller-owned buffers,
 * calls that only enqueue work on the given stream, argument errors reported
 * before anything is enqueued, the message of a failed call in
 * moe_last_error().  Nothing is allocated and no call synchronises (except
 * paged_get_device_error).  What only the GPU can see (a page number outside
 * the cache, a wait that ran past its limit) sets a bit of a device error
 * word instead of faulting.
 *
 * The cache.  A page holds `page` rows; a row holds one token's key (in the
 * `k` array) and value (in the `v` array) of every key/value head.  Sequence
 * n's token j lies in row j % page of page table[n][j / page].  Element
 * (page p, row r, head h, feature e) of k and of v is at
 *     p * page_stride + r * row_stride + h * head_stride + e   (elements),
 * so [pages][page][heads][dim] and [pages][heads][page][dim], alone or as
 * slices of an array of all layers, are both strided views.
 */
#ifndef SPARSE_MOE_BIT_GB300_PAGED_H
#define SPARSE_MOE_BIT_GB300_PAGED_H

#include <stddef.h>
#include <stdint.h>

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types.  F32 only for rope(). */
enum { PAGED_BF16 = 1, PAGED_F16 = 2, PAGED_F32 = 3 };

/* Device error word bits (paged_get_device_error). */
enum {
  PAGED_DEVERR_WAIT_TIMEOUT = 1, /* an internal wait passed its limit (the
                                    outputs of that call are not valid)     */
  PAGED_DEVERR_PAGE = 2,         /* a token's page number was outside
                                    [0, pages): rope_append did not write
                                    it, attention left its key out          */
  PAGED_DEVERR_LENGTH = 4        /* a token of rope_append stood past the
                                    width * page tokens that a row of the
                                    table holds: it was not written         */
};

/* One layer's cache.  k and v 16-byte aligned; strides in elements, multiples
 * of 8; features contiguous.  rope_append writes it, paged_attention reads. */
typedef struct paged_cache {
  void* k;
  void* v;
  int dtype; /* PAGED_BF16 or PAGED_F16 */
  int pages; /* pages in the arrays */
  int page;  /* rows of a page, >= 1 */
  int heads; /* key/value heads Hk */
  int dim;   /* features of a head D: 64, 128 or 256 */
  int64_t page_stride, row_stride, head_stride;
} paged_cache;

/* A batch of N sequences with T new tokens, packed one sequence after
 * another.  Sequence n's new tokens are cu_q[n] .. cu_q[n+1]-1; kv_len[n]
 * counts its tokens, the new ones included, so that its i-th new token stands
 * at position kv_len[n] - (cu_q[n+1] - cu_q[n]) + i.  All arrays int32, on
 * the device.  cu_q is read clamped into [0, T] and non-decreasing, a negative
 * kv_len as 0.  New tokens at negative positions (a kv_len below the number
 * of new tokens) see no key and are not written to the cache.  A row of the
 * table holds width * page tokens: rope_append writes none past them (a device
 * error bit), paged_attention reads a larger kv_len as that many. */
typedef struct paged_batch {
  const int32_t* table; /* [N][width], rows table_stride apart */
  const int32_t* cu_q;  /* [N + 1] */
  const int32_t* kv_len; /* [N] */
  int N, T, width;
  int64_t table_stride;
} paged_batch;

/*
 * Rotary positions.  With r frequencies the first 2r features of every head
 * turn, pair i by the angle pos * freq[i]; the rest pass unchanged:
 *   half layout          (a, b) = (x[i],  x[i + r])
 *   interleaved layout   (a, b) = (x[2i], x[2i + 1])
 *   a' = mscale (a cos - b sin),   b' = mscale (a sin + b cos)
 * inverse turns by the negative angle, which with the same mscale is the
 * gradient: dx = rope(dy, inverse = 1).
 *   x, out  dtype [T][H][D], token and head strides in elements (features
 *           contiguous); out may be x (in place) or must not overlap it
 *   pos     int32 [T];  freq  fp64 [r] (device), radians a position.  The
 *           angle is taken modulo one turn exactly (64-bit fixed point), so
 *           it does not lose bits at far positions.
 */
moe_status rope(const void* x, void* out, int dtype, int T, int H, int D, int64_t x_token_stride,
                int64_t x_head_stride, int64_t out_token_stride, int64_t out_head_stride,
                const int32_t* pos, const double* freq, int r, float mscale, int interleaved,
                int inverse, void* stream);

/* Frequencies of the usual scalings for long contexts (host; freq_host [rot/2],
 * *mscale the factor for cos and sin).  base_i = base^(-2i/rot) and
 *   ROPE_SCALE_NONE    base_i
 *   ROPE_SCALE_LINEAR  base_i / factor
 *   ROPE_SCALE_NTK     base_i with base * factor^(rot/(rot-2)); needs rot > 2
 *   ROPE_SCALE_YARN    between base_i / factor and base_i by a linear ramp
 *                      over i between the pairs that turn `high` (fast) and
 *                      `low` (slow) times within `original` positions;
 *                      mscale = 0.1 ln(factor) + 1 for factor > 1
 *   ROPE_SCALE_BANDED  base_i / factor below `low` turns within `original`
 *                      positions, base_i above `high`, linear in the number
 *                      of turns between
 * factor, base > 0; original, low, high are read by the last two only (0 <
 * low < high). */
enum { ROPE_SCALE_NONE = 0, ROPE_SCALE_LINEAR = 1, ROPE_SCALE_NTK = 2, ROPE_SCALE_YARN = 3,
       ROPE_SCALE_BANDED = 4 };
moe_status rope_frequencies(int rot, double base, int scaling, double factor, double original,
                            double low, double high, double* freq_host, double* mscale);

/*
 * The step before attention: turn the new tokens' queries and keys by their
 * positions in their sequences and write keys and values into the cache.
 *   q  [T][Hq][D] -> q_out (may be q: in place);  k, v [T][heads][D] -> cache
 * all of the cache's dtype, token strides in elements, heads D apart inside
 * q, k and v (a fused projection's output is three such views); q_out dense.
 * Tokens outside every sequence are not written; a token at a negative
 * position gets its q turned and no row of the cache.
 */
moe_status rope_append(const void* q, int64_t q_token_stride, void* q_out, int Hq, const void* k,
                       int64_t k_token_stride, const void* v, int64_t v_token_stride,
                       const paged_cache* cache, const paged_batch* batch, const double* freq,
                       int r, float mscale, int interleaved, void* stream);

/*
 * Attention of the new tokens over the cache (their own keys and values
 * written before).  Query head h reads key/value head h / (Hq / heads).  For
 * a query at position p >= 0, over the keys j < kv_len[n] with
 *   causal: j <= p;   window > 0: p - j < window
 *   o = sum_j softmax_j(scale q.k_j) v_j,  lse = ln sum_j exp(scale q.k_j)
 * A query that sees no key gets o = 0 and lse = -inf; the rows of o and lse of
 * tokens outside every sequence are not written.  Scores, softmax statistics
 * and sums are fp32; the weights are rounded to the cache's type (in fp16 at
 * the upper end of its range) for the product with v.  Rows of the cache at or
 * past kv_len, or whose page number is bad, may hold anything, NaN included;
 * values of visible rows are expected to be finite (a non-finite value may
 * reach queries of its chunk that do not see it).
 *   q, o   cache dtype [T][Hq][D], token and head strides in elements,
 *          multiples of 8, 16-byte aligned; must not overlap
 *   lse    fp32 [T][Hq] dense, or NULL
 *   max_q, max_kv  what the caller knows of the longest chunk and context;
 *          they choose the kernel and the split over the keys and bound
 *          nothing (0: not known; T / N and the table's width stand in)
 *   workspace  16-byte aligned, paged_attention_workspace() bytes for the
 *          same sizes (which may be 0); holds nothing between calls
 */
moe_status paged_attention_workspace(const paged_cache* cache, const paged_batch* batch, int Hq,
                                     int window, int max_q, int max_kv, size_t* bytes);
moe_status paged_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int Hq,
                           const paged_cache* cache, const paged_batch* batch, float scale,
                           int causal, int window, int max_q, int max_kv, void* o,
                           int64_t o_token_stride, int64_t o_head_stride, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * Page maintenance.  State, all int32 on the device and updated in place:
 *   refs  [P]         sequences that hold page p; 0 = free
 *   table [S][width]  pages of sequence slot s in order, rows table_stride
 *                     apart; -1 where it holds none
 *   lens  [S]         tokens of sequence slot s (0 = an empty slot)
 * The calls are deterministic: free pages are taken lowest number first.
 * Page numbers outside [0, P) in a table are passed over.
 */

/* For i < F: slot dst[i] becomes a copy of slot src[i] that shares its pages.
 * A pair is left out (and counted in *refused, int32 or NULL) when a slot is
 * out of range, dst[i] is not empty (lens != 0), an earlier pair has the same
 * dst, or src[i] is the dst of any pair. */
moe_status pages_fork(int32_t* refs, int P, int32_t* table, int64_t table_stride, int width,
                      int32_t* lens, int S, const int32_t* src, const int32_t* dst, int F,
                      int32_t* refused, void* stream);

/* Room for add[s] >= 0 more tokens in every slot (negative counts as 0); lens
 * grows by it.  A slot that grows and whose last page is partly filled and
 * shared gets a page of its own in its place (each such slot, also where all
 * that share the page grow): moves[s] = {shared page, own page}, whose rows the
 * caller copies (pages_copy) before it writes; otherwise moves[s] = {-1, -1}.
 * Pages go to slots in order of s, each slot's exchanged page first.  All or
 * nothing: status[0] = pages that were missing, status[1] = slots whose row of
 * the table is too short (or whose length would pass 2^31 - 1); where either is
 * not 0 nothing but status and moves (all -1) is written.
 * scratch: int32 [S + 1]. */
moe_status pages_reserve(int32_t* refs, int P, int32_t* table, int64_t table_stride, int width,
                         int32_t* lens, const int32_t* add, int S, int page, int32_t* moves,
                         int32_t* status, int32_t* scratch, void* stream);

/* Slots slots[i], i < F, give up their pages: refs down by one each, the row
 * of the table -1, lens 0.  Numbers out of range and repeats are left out. */
moe_status pages_free(int32_t* refs, int P, int32_t* table, int64_t table_stride, int width,
                      int32_t* lens, int S, const int32_t* slots, int F, void* stream);

/* Renumber the L pages in use to 0 .. L-1: the pages at L and above go, in
 * order, to the free numbers below L, in order.  moves [P][2] lists the pairs
 * {from, to} and then {-1, -1}; *count is their number.  refs and table are
 * updated; the pages' rows are the caller's to copy (pages_copy).
 * scratch: int32 [P + 1]. */
moe_status pages_compact(int32_t* refs, int P, int32_t* table, int64_t table_stride, int width,
                         int S, int32_t* moves, int32_t* count, int32_t* scratch, void* stream);

/* Copy page moves[i][0] to page moves[i][1], i < M, in each of B arrays of P
 * pages: array b's page p is page_bytes bytes at pools + b * pool_stride +
 * p * page_stride (bytes; pools, strides and page_bytes multiples of 16).
 * Pairs with a number outside [0, P) are left out; no page may be both read
 * and written, nor written twice.  count (device, may be NULL): only the first
 * min(M, *count) pairs. */
moe_status pages_copy(void* pools, int B, int64_t pool_stride, int P, int64_t page_stride,
                      int64_t page_bytes, const int32_t* moves, int M, const int32_t* count,
                      void* stream);

/* Synchronise `stream` and read (then clear) the current device's error word
 * of this header's calls (PAGED_DEVERR_* bits).  One word serves all streams
 * of the device; a bit that is set after the read stays for the next call. */
moe_status paged_get_device_error(void* stream, int* code);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_MOE_BIT_GB300_PAGED_H */
