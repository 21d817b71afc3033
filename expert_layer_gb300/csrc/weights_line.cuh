// The line of all sequences' work that the kernels of the keys' weights cut
// into equal ranges.
#pragma once

#include "attn.h"

namespace moe {
namespace attn {
namespace {

// Tokens and keys of a sequence; none where its entries are out of order
struct Seq {
  int q0, n, len;
};
__device__ __forceinline__ Seq seq_of(const WeightArgs& a, int s, bool& bad) {
  Seq v;
  v.q0 = a.q_starts[s];
  const int q1 = a.q_starts[s + 1];
  v.len = a.kv_lens[s];
  v.n = q1 - v.q0;
  if (v.q0 < 0 || q1 < v.q0 || q1 > a.T || v.len < 0 || v.len > a.capacity ||
      v.len > ((long long)a.table_pages << a.page_shift)) {
    bad = true;
    v.n = v.len = 0;
  }
  return v;
}

// Where ranges begin (shared memory): ranges of `each` places; of the block's
// own, up to kThreads / 32 of them, the sequence that each begins in (-1: none)
// and that sequence's first place.
template <int kThreads>
struct LineStart {
  long long scan[kThreads / 32];
  long long at[kThreads / 32];
  int seq[kThreads / 32];
  long long each;
  __device__ __forceinline__ long long begin(long long range) const { return range * each; }
};

// The grid's ranges, `per_block` for each block; weight: the places that a
// sequence takes.  Every thread sums a run of sequences.  (Ends with a barrier.)
template <int kThreads, typename Weight>
__device__ __forceinline__ void find_start(const WeightArgs& a, LineStart<kThreads>& st, int per_block, Weight weight,
                                           bool& bad) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int run = (a.n_seq + kThreads - 1) / kThreads;
  const int s0 = min(a.n_seq, (int)threadIdx.x * run), s1 = min(a.n_seq, s0 + run);
  if (threadIdx.x == 0) bad |= a.q_starts[0] != 0 || a.q_starts[a.n_seq] != a.T;
  long long mine = 0;
  for (int s = s0; s < s1; ++s) mine += weight(seq_of(a, s, bad));
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) st.scan[warp] = incl;
  if (lane == 0) st.seq[warp] = -1;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += st.scan[w];
    total += st.scan[w];
  }
  const long long ranges = (long long)gridDim.x * per_block, each = (total + ranges - 1) / ranges;
  if (threadIdx.x == 0) st.each = each;
  for (int w = 0; w < per_block; ++w) {
    const long long at = ((long long)blockIdx.x * per_block + w) * each;
    if (at < before || at >= before + mine) continue;
    long long p = before;
    for (int s = s0; s < s1; ++s) {
      const long long n = weight(seq_of(a, s, bad));
      if (at < p + n) {
        st.seq[w] = s;
        st.at[w] = p;
        break;
      }
      p += n;
    }
  }
  __syncthreads();
}

}  // namespace
}  // namespace attn
}  // namespace moe
