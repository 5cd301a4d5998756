// The groups of a batch whose sequences share their first keys, as a batch of their own
// (include/paged.h, paged_attention_shared).
#include "paged_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kFew = 8;  // tokens of a sequence that one thread maps

// A CTA a group.  What a group can share: no more than its members all have before their
// new tokens, so that every one of these keys is visible to all of its rows, and nothing
// where fewer than two of them have new tokens.
__global__ void __launch_bounds__(kThreads) groups_kernel(const BatchView b, const GroupView g) {
  __shared__ int sh_first, sh_least, sh_with, sh_at;
  // the attention over the shared keys may be set up meanwhile
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int me = blockIdx.x;
  if (threadIdx.x == 0) {
    sh_first = b.N;
    sh_least = 0x7fffffff;
    sh_with = 0;
    sh_at = 0;
  }
  __syncthreads();
  // cu_group made non-decreasing within [0, N]
  for (int i = threadIdx.x; i <= me; i += kThreads) atomicMax(&sh_at, min(g.cu_group[i], b.N));
  __syncthreads();
  const int n0 = sh_at, n1 = min(max(g.cu_group[me + 1], n0), b.N);
  for (int n = n0 + threadIdx.x; n < n1; n += kThreads) {
    const Seq s = load_seq(b, n);
    if (s.nq == 0) continue;
    atomicMin(&sh_first, n);
    atomicMin(&sh_least, s.kv - s.nq);
    atomicAdd(&sh_with, 1);
  }
  __syncthreads();
  const int len = sh_with < 2 ? 0 : max(min(g.shared[me], sh_least), 0);
  // the first and the last group's CTA also take the sequences of no group
  const int a0 = me == 0 ? 0 : n0, a1 = me == g.G - 1 ? b.N : n1;
  const int lane = threadIdx.x & 31;
  for (int base = a0 + (int)threadIdx.x - lane; base < a1; base += kThreads) {
    const int n = base + lane, at = g.own + n;
    const bool there = n < a1, in = n >= n0 && n < n1;
    const Seq s = load_seq(b, min(n, b.N - 1));
    const int group = in ? me : -1;
    if (there) {
      g.skip[at] = in ? len : 0;
      if (g.own) {
        g.cu[at] = b.cu[n];
        if (n == b.N - 1) g.cu[at + 1] = b.cu[n + 1];
        g.len[at] = b.kv_len[n];
        g.rows[at] = n;
      }
    }
    // a sequence's tokens: a few by its own thread, a chunk's by the warp (a call over one of
    // 8192: 467 us, 502 with a thread for all)
    const bool chunk = there && s.nq > kFew;
    if (there && !chunk)
      for (int t = s.t0; t < s.t0 + s.nq; ++t) g.of_token[t] = make_int2(at, group);
    for (unsigned left = __ballot_sync(0xffffffffu, chunk); left; left &= left - 1) {
      const int src = __ffs((int)left) - 1;
      const int t0 = __shfl_sync(0xffffffffu, s.t0, src), t1 = t0 + __shfl_sync(0xffffffffu, s.nq, src);
      const int2 of = make_int2(g.own + base + src, __shfl_sync(0xffffffffu, group, src));
      for (int t = t0 + lane; t < t1; t += 32) g.of_token[t] = of;
    }
  }
  if (threadIdx.x == 0) {
    g.len[me] = len;
    g.rows[me] = min(sh_first, b.N - 1);
    g.cu[me] = b.cu[n0];
    if (me == g.G - 1) g.cu[g.G] = b.cu[n1];
    if (g.own) {
      g.skip[me] = 0;
      if (me == g.G - 1) g.len[g.G] = g.rows[g.G] = g.skip[g.G] = 0;
    }
  }
}

}  // namespace

cudaError_t launch_paged_groups(const BatchView& b, const GroupView& g, cudaStream_t st) {
  return launch_kernel(groups_kernel, dim3(g.G), dim3(kThreads), 0, st, b, g);
}

}  // namespace moe
