// Query / key norms, rotary positions and the append to the paged cache.
//
// For every row (token t, head h) of the projection, fp32 throughout:
//   n(x)_i = x_i w_i / sqrt(sum x^2 / D + eps)
//   (a, b) -> (a cos - b sin, b cos + a sin) for the pairs of the first rot
//   elements: (i, i + rot/2), or (2i, 2i + 1) interleaved
// and q goes to q_out, k and v to the cache row of the token's slot.
//
// Bound: HBM.  A row is read once and written once (4 D bytes) for ~8 D
// flops.  A row is held by D/8 lanes of one warp, 16 bytes each, so the norm
// is a shuffle sum and the partner of a half-layout pair one shuffle away.
#include "attn.h"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = 256;

template <bool kF16>
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (kF16) {
      asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}"
          : "=f"(x[2 * j]), "=f"(x[2 * j + 1])
          : "r"(w[j]));
    } else {
      x[2 * j] = bf16lo(w[j]);
      x[2 * j + 1] = bf16hi(w[j]);
    }
  }
}

template <bool kF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (kF16) w[j] = (uint32_t)f2h(x[2 * j]) | ((uint32_t)f2h(x[2 * j + 1]) << 16);
    else w[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A group of D/8 lanes takes items of one token and kHeads consecutive heads
// (of the Hq + 2 Hkv heads of q, k and v); lane i of the group holds elements
// 8i .. 8i+7 of each row.
template <int D, int kHeads, bool kF16>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeArgs a, const Report rep) {
  constexpr int kLanes = D / 8, kGroups = kThreads / kLanes;
  const int gl = threadIdx.x % kLanes;                 // lane of the group
  const int heads = a.Hq + 2 * a.Hkv;
  const int chunks = (heads + kHeads - 1) / kHeads;
  const long long items = (long long)a.T * chunks;
  const int half = a.rot / 2;
  bool bad = false;
  float wq[8], wk[8];                                  // this lane's norm weights
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    wq[j] = a.q_norm ? a.q_norm[8 * gl + j] : 1.0f;
    wk[j] = a.k_norm ? a.k_norm[8 * gl + j] : 1.0f;
  }
  // the loop's trip count is the same for the lanes of a warp: shuffles below
  for (long long base = (long long)blockIdx.x * kGroups; base < items; base += (long long)gridDim.x * kGroups) {
    const long long item = base + threadIdx.x / kLanes;
    const bool live = item < items;
    const int t = live ? (int)(item / chunks) : 0;
    const int h0 = live ? (int)(item % chunks) * kHeads : 0;
    int pos = a.positions[t];
    const int slot = a.slots[t];
    bool ok = live;
    if ((unsigned)pos >= (unsigned)a.max_pos) {
      bad |= live;
      ok = false;
      pos = 0;
    }
    const bool slot_ok = slot >= 0 && (slot >> a.page_shift) < a.pages;
    if (slot >= 0 && !slot_ok) bad |= live;
    // this lane's angles: elements 8 gl .. of the half layout use angle
    // (8 gl + j) mod half; pairs 4 gl + j of the interleaved one
    float cs[8], sn[8];
    const bool turns = 8 * gl < a.rot;
    if (turns) {
      const float* row = a.table + (long long)pos * a.rot;
      if (a.interleaved) {
        const float4 c = *reinterpret_cast<const float4*>(row + 4 * gl);
        const float4 s = *reinterpret_cast<const float4*>(row + half + 4 * gl);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          cs[j] = cc[j / 2];
          sn[j] = (j & 1) ? ss[j / 2] : -ss[j / 2];
        }
      } else {
        const bool first = 8 * gl < half;
        const float* p = row + 8 * gl - (first ? 0 : half);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          cs[j] = p[j];
          sn[j] = first ? -p[half + j] : p[half + j];
        }
      }
    }
    const int partner = !turns ? gl : 8 * gl < half ? gl + half / 8 : gl - half / 8;
    uint4 raw[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = h0 + i;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (live && h < heads) {
        const Heads& src = h < a.Hq ? a.q : h < a.Hq + a.Hkv ? a.k : a.v;
        const int hh = h < a.Hq ? h : h < a.Hq + a.Hkv ? h - a.Hq : h - a.Hq - a.Hkv;
        raw[i] = *reinterpret_cast<const uint4*>(src.data + t * src.tok + hh * src.head + 8 * gl);
      }
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = h0 + i;
      const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
      uint4 o = raw[i];
      float x[8];
      unpack8<kF16>(raw[i], x);
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
      for (int d = 1; d < kLanes; d <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d, kLanes);
      if (is_q ? a.q_norm != nullptr : a.k_norm != nullptr) {
        const float r = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= r * (is_q ? wq[j] : wk[j]);
      }
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        y[j] = a.interleaved ? x[j ^ 1] : __shfl_sync(0xffffffffu, x[j], partner, kLanes);
      if (turns)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fmaf(y[j], sn[j], x[j] * cs[j]);
      if (!is_v) o = pack8<kF16>(x);
      if (!ok || h >= heads) continue;
      if (is_q) {
        *reinterpret_cast<uint4*>(a.q_out + ((long long)t * a.Hq + h) * D + 8 * gl) = o;
      } else if (slot_ok) {
        const int hh = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
        const long long page = slot >> a.page_shift, row = slot & ((1 << a.page_shift) - 1);
        uint16_t* c = is_v ? a.v_cache : a.k_cache;
        *reinterpret_cast<uint4*>(c + (((page * a.Hkv + hh) << a.page_shift) + row) * D + 8 * gl) = o;
      }
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) report(rep, any ? kStatusBounds : 0);
}

template <int D, int kHeads, bool kF16>
cudaError_t launch(const RopeArgs& a, void* ws, int num_sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  const int chunks = (a.Hq + 2 * a.Hkv + kHeads - 1) / kHeads;
  const long long blocks = ((long long)a.T * chunks + kGroups - 1) / kGroups;
  const long long most = (long long)num_sms * 8 < kFlagsPerSet ? (long long)num_sms * 8 : kFlagsPerSet;
  const int grid = (int)(blocks < most ? blocks : most);
  const Report rep{ws, 0, {grid, 0}};
  rope_append_kernel<D, kHeads, kF16><<<grid, kThreads, 0, stream>>>(a, rep);
  return cudaGetLastError();
}

template <int D, int kHeads>
cudaError_t launch_type(const RopeArgs& a, void* ws, int num_sms, cudaStream_t stream) {
  return a.f16 ? launch<D, kHeads, true>(a, ws, num_sms, stream) : launch<D, kHeads, false>(a, ws, num_sms, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, void* ws, int num_sms, cudaStream_t stream) {
  // four heads to a group once that still gives every SM a full set of threads
  const bool many = (long long)a.T * (a.Hq + 2 * a.Hkv) * (a.D / 8) / 4 >= 1024ll * num_sms;
  if (a.D == 64) return many ? launch_type<64, 4>(a, ws, num_sms, stream) : launch_type<64, 1>(a, ws, num_sms, stream);
  return many ? launch_type<128, 4>(a, ws, num_sms, stream) : launch_type<128, 1>(a, ws, num_sms, stream);
}

}  // namespace attn
}  // namespace moe
