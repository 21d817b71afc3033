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
// and ends in 7 us).
#include "attn.h"
#include "attn_ptx.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kMany = 4;            // heads per group of lanes once there are enough of them
constexpr int kResident = 4;        // blocks of an SM, all that run: 64 registers a thread

// Two elements to fp32 and back
template <bool kF16>
__device__ __forceinline__ uint64_t unpack2(uint32_t w) {
  float x, y;
  if (kF16) {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}"
        : "=f"(x), "=f"(y)
        : "r"(w));
  } else {
    x = bf16lo(w);
    y = bf16hi(w);
  }
  return pair(x, y);
}

// Four consecutive elements
struct Part {
  uint32_t w[2];
  __device__ __forceinline__ void load(const uint16_t* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]); }
};

// Items: (token, kHeads consecutive heads of q, of k or of v).
template <int D, int kHeads, bool kF16, bool kInter>
__global__ void __launch_bounds__(kThreads, kResident)
    rope_append_kernel(const RopeArgs a, const Report rep) {
  constexpr int kPart = 4, kLanes = D / (2 * kPart), kGroups = kThreads / kLanes;
  const int gl = threadIdx.x % kLanes;                  // lane of the group
  const unsigned cq = (a.Hq + kHeads - 1) / kHeads, ck = (a.Hkv + kHeads - 1) / kHeads, chunks = a.chunks;
  const unsigned long long items = (unsigned long long)a.T * chunks;
  const int half = a.rot / 2;
  const bool turns = 2 * kPart * gl < a.rot;
  const int o1 = kInter || !turns ? 2 * kPart * gl : kPart * gl, o2 = kInter || !turns ? o1 + kPart : half + o1;
  const bool norms = a.q_norm || a.k_norm;
  bool bad = false;
  // the trip count is the same for the lanes of a warp: shuffles below
  for (unsigned long long base = (unsigned long long)blockIdx.x * kGroups; base < items;
       base += (unsigned long long)gridDim.x * kGroups) {
    const unsigned long long item = base + threadIdx.x / kLanes;
    const bool live = item < items;
    const unsigned long long it = live ? item : 0;
    const unsigned t = items >> 31 ? (unsigned)(it / chunks) : (unsigned)a.by_chunks.of((int)it);
    const unsigned chunk = (unsigned)(it - (unsigned long long)t * chunks);
    int pos = a.positions[t];
    const int slot = a.slots[t];
    const int kind = chunk < cq ? 0 : chunk < cq + ck ? 1 : 2;            // q, k, v
    const int h0 = (int)(chunk - (kind == 0 ? 0 : kind == 1 ? cq : cq + ck)) * kHeads;
    const int n = live ? min(kHeads, (kind == 0 ? a.Hq : a.Hkv) - h0) : 0;
    const Heads& src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const uint16_t* in = src.data + t * src.tok + h0 * src.head;
    const long long in_step = src.head;
    Part raw[kHeads][2];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
      if (i < n) {
        raw[i][0].load(in + i * in_step + o1);
        raw[i][1].load(in + i * in_step + o2);
      } else {
        raw[i][0] = raw[i][1] = Part{};
      }
    bool ok = live;
    if ((unsigned)pos >= (unsigned)a.max_pos) {
      bad |= live;
      ok = false;
      pos = 0;
    }
    const bool slot_ok = slot >= 0 && (slot >> a.page_shift) < a.pages;
    if (slot >= 0 && !slot_ok) bad |= live;
    uint16_t* out = a.q_out + ((long long)t * a.Hq + h0) * D;
    long long out_step = D;
    if (kind) {
      const long long page = slot >> a.page_shift, row = slot & ((1 << a.page_shift) - 1);
      out = (kind == 1 ? a.k_cache : a.v_cache) + (((page * a.Hkv + h0) << a.page_shift) + row) * D;
      out_step = (long long)D << a.page_shift;
      ok = ok && slot_ok;
    }
    const float* weight = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
    // coefficients: y_j = x_j c_j + partner(x_j) s_j
    float c[2 * kPart], s[2 * kPart];
#pragma unroll
    for (int j = 0; j < 2 * kPart; ++j) c[j] = weight ? weight[(j < kPart ? o1 : o2) + j % kPart] : 1.0f, s[j] = 0.f;
    if (turns) {
      const float* row = a.table + (long long)pos * a.rot + kPart * gl;
      const float4 cc = *reinterpret_cast<const float4*>(row), ss = *reinterpret_cast<const float4*>(row + half);
      const float co[4] = {cc.x, cc.y, cc.z, cc.w}, si[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
      for (int j = 0; j < kPart; ++j) {
        const int p = kInter ? 2 * j : j, q = kInter ? p + 1 : p + kPart;   // the pair's two elements
        s[p] = -si[j] * c[q];
        s[q] = si[j] * c[p];
        c[p] *= co[j];
        c[q] *= co[j];
      }
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      uint64_t x[kPart];             // pairs of neighbours
      float r = 1.0f;
#pragma unroll
      for (int j = 0; j < kPart; ++j) x[j] = unpack2<kF16>(raw[i][j / (kPart / 2)].w[j % (kPart / 2)]);
      if (norms) {
        uint64_t sum2 = 0;
#pragma unroll
        for (int j = 0; j < kPart; ++j) sum2 = fma2(x[j], x[j], sum2);
        float sum = lo(sum2) + hi(sum2);
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d, kLanes);
        if (weight) r = rsqrtf(fmaf(sum, 1.0f / D, a.eps));
      }
      Part y[2];
      const uint64_t r2 = pair(r, r);
#pragma unroll
      for (int j = 0; j < kPart; ++j) {
        uint64_t v = mul2(x[j], pair(c[2 * j], c[2 * j + 1]));
        // (an element that is not rotated has no other whose infinity it would take on)
        if (turns)
          v = fma2(kInter ? pair(hi(x[j]), lo(x[j])) : x[(j + kPart / 2) % kPart], pair(s[2 * j], s[2 * j + 1]), v);
        v = mul2(v, r2);
        y[j / (kPart / 2)].w[j % (kPart / 2)] = pack2<kF16>(lo(v), hi(v));
      }
      if (!ok || i >= n) continue;
      uint16_t* dst = out + i * out_step;
      (kind == 2 ? raw[i][0] : y[0]).store(dst + o1);
      (kind == 2 ? raw[i][1] : y[1]).store(dst + o2);
    }
  }
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
  if (a.interleaved) rope_append_kernel<D, kHeads, kF16, true><<<grid, kThreads, 0, stream>>>(a, rep);
  else rope_append_kernel<D, kHeads, kF16, false><<<grid, kThreads, 0, stream>>>(a, rep);
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
