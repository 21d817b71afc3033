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
#include "attn.h"
#include "attn_ptx.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = 256;

template <bool kF16>
__device__ __forceinline__ void unpack4(uint2 v, float* x) {
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
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
__device__ __forceinline__ uint2 pack4(const float* x) {
  return make_uint2(pack2<kF16>(x[0], x[1]), pack2<kF16>(x[2], x[3]));
}

// Items: (token, kHeads consecutive heads of q, of k or of v).
template <int D, int kHeads, bool kF16, bool kInter>
__global__ void __launch_bounds__(kThreads, kHeads > 1 ? 4 : 1) rope_append_kernel(const RopeArgs a, const Report rep) {
  constexpr int kLanes = D / 8, kGroups = kThreads / kLanes;
  constexpr int kBatch = kHeads < 4 ? kHeads : 4;       // rows whose loads are in flight together
  const int gl = threadIdx.x % kLanes;                  // lane of the group
  const unsigned cq = (a.Hq + kHeads - 1) / kHeads, ck = (a.Hkv + kHeads - 1) / kHeads, chunks = cq + 2 * ck;
  const unsigned long long items = (unsigned long long)a.T * chunks;
  const int half = a.rot / 2;
  const bool turns = 8 * gl < a.rot;
  const int o1 = kInter ? 8 * gl : turns ? 4 * gl : 8 * gl, o2 = kInter || !turns ? o1 + 4 : half + 4 * gl;
  const bool norms = a.q_norm || a.k_norm;
  bool bad = false;
  // the trip count is the same for the lanes of a warp: shuffles below
  for (unsigned long long base = (unsigned long long)blockIdx.x * kGroups; base < items;
       base += (unsigned long long)gridDim.x * kGroups) {
    const unsigned long long item = base + threadIdx.x / kLanes;
    const bool live = item < items;
    const unsigned long long it = live ? item : 0;
    const unsigned t = items >> 32 ? (unsigned)(it / chunks) : (unsigned)it / chunks;
    const unsigned chunk = (unsigned)(it - (unsigned long long)t * chunks);
    int pos = a.positions[t];
    const int slot = a.slots[t];
    const int kind = chunk < cq ? 0 : chunk < cq + ck ? 1 : 2;            // q, k, v
    const int h0 = (int)(chunk - (kind == 0 ? 0 : kind == 1 ? cq : cq + ck)) * kHeads;
    const int n = live ? min(kHeads, (kind == 0 ? a.Hq : a.Hkv) - h0) : 0;
    const Heads& src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const uint16_t* in = src.data + t * src.tok + h0 * src.head;
    const long long in_step = src.head;
    uint2 raw[kBatch][2];
    auto load = [&](int i0) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i0 + i < n) {
          raw[i][0] = *reinterpret_cast<const uint2*>(in + (i0 + i) * in_step + o1);
          raw[i][1] = *reinterpret_cast<const uint2*>(in + (i0 + i) * in_step + o2);
        } else {
          raw[i][0] = raw[i][1] = make_uint2(0, 0);
        }
    };
    load(0);
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
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = weight ? weight[(j < 4 ? o1 : o2) + (j & 3)] : 1.0f;
    if (turns) {
      const float* row = a.table + (long long)pos * a.rot + 4 * gl;
      const float4 cc = *reinterpret_cast<const float4*>(row), ss = *reinterpret_cast<const float4*>(row + half);
      const float co[4] = {cc.x, cc.y, cc.z, cc.w}, si[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = kInter ? 2 * j : j, q = kInter ? 2 * j + 1 : j + 4;   // the pair's two elements
        s[p] = -si[j] * c[q];
        s[q] = si[j] * c[p];
        c[p] *= co[j];
        c[q] *= co[j];
      }
    }
#pragma unroll
    for (int i0 = 0; i0 < kHeads; i0 += kBatch) {
      if (i0) load(i0);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        float x[8], y[8], r = 1.0f;
        unpack4<kF16>(raw[i][0], x);
        unpack4<kF16>(raw[i][1], x + 4);
        if (norms) {
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
          for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d, kLanes);
          if (weight) r = rsqrtf(fmaf(sum, 1.0f / D, a.eps));
        }
        if (turns) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = fmaf(x[kInter ? j ^ 1 : j ^ 4], s[j], x[j] * c[j]) * r;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = x[j] * c[j] * r;
        }
        if (!ok || i0 + i >= n) continue;
        uint16_t* dst = out + (i0 + i) * out_step;
        *reinterpret_cast<uint2*>(dst + o1) = kind == 2 ? raw[i][0] : pack4<kF16>(y);
        *reinterpret_cast<uint2*>(dst + o2) = kind == 2 ? raw[i][1] : pack4<kF16>(y + 4);
      }
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) report(rep, blockIdx.x, any ? kStatusBounds : 0);
}

template <int D, int kHeads, bool kF16>
cudaError_t launch(const RopeArgs& a, void* ws, int num_sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  const long long chunks = (a.Hq + kHeads - 1) / kHeads + 2 * ((a.Hkv + kHeads - 1) / kHeads);
  const long long blocks = (a.T * chunks + kGroups - 1) / kGroups;
  const long long most = (long long)num_sms * 8 < kFlagsFirst ? (long long)num_sms * 8 : kFlagsFirst;
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
  // eight heads to a group once that still gives every SM a full set of threads
  const bool many = (long long)a.T * (a.Hq + 2 * a.Hkv) * (a.D / 8) / 8 >= 1024ll * num_sms;
  if (a.D == 64) return many ? launch_type<64, 8>(a, ws, num_sms, stream) : launch_type<64, 1>(a, ws, num_sms, stream);
  return many ? launch_type<128, 8>(a, ws, num_sms, stream) : launch_type<128, 1>(a, ws, num_sms, stream);
}

}  // namespace attn
}  // namespace moe
