// Query / key norms, rotary positions and the append to the paged cache.
//
// For every row (token t, head h) of the projection, fp32 throughout:
//   n(x)_i = x_i w_i / sqrt(sum x^2 / D + eps)
//   (a, b) -> (a cos - b sin, b cos + a sin) for the pairs of the first rot
//   elements: (i, i + rot/2), or (2i, 2i + 1) interleaved
// and q goes to q_out, k and v to the cache row of the token's slot.
//
// Bound: HBM for many tokens (a row is read once and written once, 4 D bytes
// for ~8 D flops), latency for few.  A row is held by a group of D/8 lanes,
// each with both elements of its pairs, so that rotating takes no exchange:
// lane i has elements 4i .. 4i+3 and rot/2 + 4i .. of the half layout (8 of
// the unrotated rest for lanes from rot/8 on), 8i .. 8i+7 of the interleaved
// one; the angles of both are 4i .. 4i+3.  A group takes several heads of one
// token, for which cos, sin and the norm's weights are combined once:
//   a' = r (a (w_a cos) - b (w_b sin)),  b' = r (b (w_b cos) + a (w_a sin)),
//   r = 1 / sqrt(mean x^2 + eps)
// The grid is what the GPU holds at once (twice that: 8192 tokens of 32 + 2 x 4
// heads of 128, 33.0 us instead of 32.4), four heads to a group (eight: 32.0,
// but 64-wide heads 19.4 instead of 18.0 us), four elements to a load (eight,
// with half the lanes and twice the registers: 36.9).
// Measured: 1 token 2.2 us, 256 tokens 3.3, 8192 tokens 32.1 us = 5.4 TB/s, 79%
// of a copy's rate; 16,384 tokens 59.4 us = 5.8 TB/s (a call of 172 MB starts
// and ends in 7 us).  Positions of three axes: 4096 tokens 17.2 us, 64 (12 + 2 x 3
// heads of 64) 2.7.
#include "attn.h"
#include "attn_ptx.cuh"
#include "rope_rows.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = kRopeThreads;
constexpr int kMany = 4;            // heads per group of lanes once there are enough of them
constexpr int kResident = 4;        // blocks of an SM, all that run: 64 registers a thread

template <int D, int kHeads, bool kF16, bool kInter, bool kAxes>
__global__ void __launch_bounds__(kThreads, kResident)
    rope_append_kernel(const RopeArgs a, const Report rep) {
  const bool bad = rope_rows<D, kHeads, kF16, kInter, true>(a, kAxes, blockIdx.x, gridDim.x);
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) report(rep, blockIdx.x, any ? kStatusBounds : 0);
}

template <int D, int kHeads, bool kF16>
cudaError_t launch(RopeArgs a, void* ws, int num_sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  a.chunks = (a.Hq + kHeads - 1) / kHeads + 2 * ((a.Hkv + kHeads - 1) / kHeads);
  a.by_chunks.set(a.chunks);
  const long long blocks = ((long long)a.T * a.chunks + kGroups - 1) / kGroups;
  const long long most = (long long)num_sms * kResident < kFlagsFirst ? (long long)num_sms * kResident : kFlagsFirst;
  const int grid = (int)(blocks < most ? blocks : most);
  const Report rep{ws, 0, {grid, 0}};
  auto kern = a.axes ? (a.interleaved ? rope_append_kernel<D, kHeads, kF16, true, true>
                                      : rope_append_kernel<D, kHeads, kF16, false, true>)
                     : (a.interleaved ? rope_append_kernel<D, kHeads, kF16, true, false>
                                      : rope_append_kernel<D, kHeads, kF16, false, false>);
  kern<<<grid, kThreads, 0, stream>>>(a, rep);
  return cudaGetLastError();
}

template <int D, int kHeads>
cudaError_t launch_type(const RopeArgs& a, void* ws, int num_sms, cudaStream_t stream) {
  return a.f16 ? launch<D, kHeads, true>(a, ws, num_sms, stream) : launch<D, kHeads, false>(a, ws, num_sms, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, void* ws, int num_sms, cudaStream_t stream) {
  // several heads to a group once that still gives every SM 512 threads (1024
  // tokens of 32 + 2 x 4 heads 7.5 -> 5.5 us; with one head for 512 tokens
  // 4.7, several 4.05)
  const bool many = (long long)a.T * (a.Hq + 2 * a.Hkv) * (a.D / 8) / kMany >= 512ll * num_sms;
  if (a.D == 64)
    return many ? launch_type<64, kMany>(a, ws, num_sms, stream) : launch_type<64, 1>(a, ws, num_sms, stream);
  return many ? launch_type<128, kMany>(a, ws, num_sms, stream) : launch_type<128, 1>(a, ws, num_sms, stream);
}

}  // namespace attn
}  // namespace moe
