// Joins the parts of rows whose keys were split over blocks: with part i's
// result o_i and log2-sum lse_i,
//   out = sum_i w_i o_i / sum_i w_i,  w_i = 2^{lse_i - max lse},
//   lse = max lse + log2 sum_i w_i.
// A warp per row; a part without keys has lse_i = -inf and is not read.
#include "attn.h"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = 128;

template <int D, bool kF16>
__global__ void __launch_bounds__(kThreads) attn_merge_kernel(const AttnArgs a, int splits,
                                                              const float* __restrict__ part_o,
                                                              const float* __restrict__ part_lse) {
  constexpr int N = D / 32;
  pdl_wait();   // programmatic dependent launch: the parts are complete
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)a.T * a.Hq;
  const long long r = (long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (r >= rows) return;
  float top = -INFINITY;
  for (int i = 0; i < splits; ++i) top = fmaxf(top, part_lse[i * rows + r]);
  float o[N], sum = 0.f;
#pragma unroll
  for (int u = 0; u < N; ++u) o[u] = 0.f;
  if (top != -INFINITY)
    for (int i = 0; i < splits; ++i) {
      const float w = exp2f(part_lse[i * rows + r] - top);
      if (w == 0.f) continue;
      sum += w;
      const float* p = part_o + (i * rows + r) * D + lane * N;
#pragma unroll
      for (int u = 0; u < N; ++u) o[u] = fmaf(w, p[u], o[u]);
    }
  const float inv = sum > 0.f ? 1.0f / sum : sum;     // no keys: 0; NaN stays
#pragma unroll
  for (int u = 0; u < N; ++u) a.out[r * D + lane * N + u] = kF16 ? f2h(o[u] * inv) : f2bf(o[u] * inv);
  if (a.lse && lane == 0) a.lse[r] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945f;
}

}  // namespace

cudaError_t launch_attn_merge(const AttnArgs& a, int splits, const float* part_o, const float* part_lse,
                              cudaStream_t stream) {
  const long long rows = (long long)a.T * a.Hq;
  const unsigned grid = (unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32));
  auto kern = a.D == 64 ? (a.f16 ? attn_merge_kernel<64, true> : attn_merge_kernel<64, false>)
                        : (a.f16 ? attn_merge_kernel<128, true> : attn_merge_kernel<128, false>);
  return launch_pdl(kern, dim3(grid), dim3(kThreads), 0, stream, a, splits, part_o, part_lse);
}

}  // namespace attn
}  // namespace moe
