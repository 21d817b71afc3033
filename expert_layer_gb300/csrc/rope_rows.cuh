// Normed and rotated rows of a projection: what the append kernels share.
//
// A row (token t, head h) is held by a group of D/8 lanes, each with both
// elements of its pairs: lane i has elements 4i .. 4i+3 and rot/2 + 4i .. of
// the half layout (8 of the unrotated rest for lanes from rot/8 on), 8i ..
// 8i+7 of the interleaved one; the angles of both are 4i .. 4i+3.
#pragma once

#include "attn.h"
#include "attn_ptx.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kPart = 4;              // elements of a load; a lane has two of them

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

// Where lane `gl` of a group has its elements
template <bool kInter>
struct LanePlace {
  int gl, o1, o2;
  bool turns;
  __device__ __forceinline__ LanePlace(const RopeArgs& a, int lane) : gl(lane) {
    turns = 2 * kPart * gl < a.rot;
    o1 = kInter || !turns ? 2 * kPart * gl : kPart * gl;
    o2 = kInter || !turns ? o1 + kPart : a.rot / 2 + o1;
  }
};

// Positions of a token, one or (axes) one for each of a.n_axes
struct Places {
  int p[kMaxAxes];
  // false: one of them is out of range
  __device__ __forceinline__ bool load(const RopeArgs& a, bool axes, unsigned t) {
    p[0] = a.positions[t];
    bool ok = (unsigned)p[0] < (unsigned)a.max_pos;
    if (axes)
#pragma unroll
      for (int i = 1; i < kMaxAxes; ++i) {
        p[i] = i < a.n_axes ? a.positions[(long long)i * a.T + t] : 0;
        ok = ok && (unsigned)p[i] < (unsigned)a.max_pos;
      }
    return ok;
  }
};
// The axes of the lane's four pairs, a byte each; false: one is out of range
template <bool kInter>
__device__ __forceinline__ bool lane_axes(const RopeArgs& a, bool axes, const LanePlace<kInter>& at, uint32_t& which) {
  which = 0;
  if (!axes || !at.turns) return true;
  which = *reinterpret_cast<const uint32_t*>(a.axes + kPart * at.gl);
  bool ok = true;
#pragma unroll
  for (int j = 0; j < kPart; ++j) ok = ok && (int)((which >> (8 * j)) & 255) < a.n_axes;
  if (!ok) which = 0;
  return ok;
}

// Coefficients: y_j = x_j c_j + partner(x_j) s_j, the norm's weights in them
template <bool kInter>
__device__ __forceinline__ void coefficients(const RopeArgs& a, bool axes, const LanePlace<kInter>& at, uint32_t which,
                                             const Places& pos, const float* weight, float (&c)[2 * kPart],
                                             float (&s)[2 * kPart]) {
#pragma unroll
  for (int j = 0; j < 2 * kPart; ++j) c[j] = weight ? weight[(j < kPart ? at.o1 : at.o2) + j % kPart] : 1.0f, s[j] = 0.f;
  if (!at.turns) return;
  float co[kPart], si[kPart];
  if (axes) {
#pragma unroll
    for (int j = 0; j < kPart; ++j) {
      const uint32_t x = (which >> (8 * j)) & 255;
      const int p = x == 0 ? pos.p[0] : x == 1 ? pos.p[1] : x == 2 ? pos.p[2] : pos.p[3];
      const float* row = a.table + (long long)p * a.rot + kPart * at.gl + j;
      co[j] = row[0];
      si[j] = row[a.rot / 2];
    }
  } else {
    const float* row = a.table + (long long)pos.p[0] * a.rot + kPart * at.gl;
    const float4 cc = *reinterpret_cast<const float4*>(row), ss = *reinterpret_cast<const float4*>(row + a.rot / 2);
    co[0] = cc.x, co[1] = cc.y, co[2] = cc.z, co[3] = cc.w;
    si[0] = ss.x, si[1] = ss.y, si[2] = ss.z, si[3] = ss.w;
  }
#pragma unroll
  for (int j = 0; j < kPart; ++j) {
    const int p = kInter ? 2 * j : j, q = kInter ? p + 1 : p + kPart;   // the pair's two elements
    s[p] = -si[j] * c[q];
    s[q] = si[j] * c[p];
    c[p] *= co[j];
    c[q] *= co[j];
  }
}

// The lane's elements of one row, as pairs of neighbours (every lane of the
// warp takes part: the norm's sum is a shuffle)
template <int D, bool kF16, bool kInter>
__device__ __forceinline__ void turn(const Part (&raw)[2], bool norms, bool weighted, float eps, bool turns,
                                     const float (&c)[2 * kPart], const float (&s)[2 * kPart], uint64_t (&y)[kPart]) {
  constexpr int kLanes = D / (2 * kPart);
  uint64_t x[kPart];
  float r = 1.0f;
#pragma unroll
  for (int j = 0; j < kPart; ++j) x[j] = unpack2<kF16>(raw[j / (kPart / 2)].w[j % (kPart / 2)]);
  if (norms) {
    uint64_t sum2 = 0;
#pragma unroll
    for (int j = 0; j < kPart; ++j) sum2 = fma2(x[j], x[j], sum2);
    float sum = lo(sum2) + hi(sum2);
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d, kLanes);
    if (weighted) r = rsqrtf(fmaf(sum, 1.0f / D, eps));
  }
  const uint64_t r2 = pair(r, r);
#pragma unroll
  for (int j = 0; j < kPart; ++j) {
    uint64_t v = mul2(x[j], pair(c[2 * j], c[2 * j + 1]));
    // (an element that is not rotated has no other whose infinity it would take on)
    if (turns)
      v = fma2(kInter ? pair(hi(x[j]), lo(x[j])) : x[(j + kPart / 2) % kPart], pair(s[2 * j], s[2 * j + 1]), v);
    y[j] = mul2(v, r2);
  }
}

// Rows of a call, (token, kHeads consecutive heads of q, and with kCache of k
// and of v) for each group of lanes of block `block` of `blocks`: to q_out and
// the cache.  Whether an index was out of range.
template <int D, int kHeads, bool kF16, bool kInter, bool kCache>
__device__ __forceinline__ bool rope_rows(const RopeArgs& a, const bool axes, const unsigned block,
                                          const unsigned blocks) {
  constexpr int kLanes = D / (2 * kPart), kGroups = kRopeThreads / kLanes;
  const unsigned cq = (a.Hq + kHeads - 1) / kHeads, ck = (a.Hkv + kHeads - 1) / kHeads, chunks = a.chunks;
  const unsigned long long items = (unsigned long long)a.T * chunks;
  const LanePlace<kInter> at(a, threadIdx.x % kLanes);
  uint32_t which;
  bool bad = !lane_axes(a, axes, at, which);
  const bool norms = a.q_norm || (kCache && a.k_norm);
  // the trip count is the same for the lanes of a warp: shuffles below
  for (unsigned long long base = (unsigned long long)block * kGroups; base < items;
       base += (unsigned long long)blocks * kGroups) {
    const unsigned long long item = base + threadIdx.x / kLanes;
    const bool live = item < items;
    const unsigned long long it = live ? item : 0;
    const unsigned t = items >> 31 ? (unsigned)(it / chunks) : (unsigned)a.by_chunks.of((int)it);
    const unsigned chunk = (unsigned)(it - (unsigned long long)t * chunks);
    Places pos;
    const bool placed = pos.load(a, axes, t);
    const int slot = kCache ? a.slots[t] : 0;
    const int kind = !kCache || chunk < cq ? 0 : chunk < cq + ck ? 1 : 2;            // q, k, v
    const int h0 = (int)(chunk - (kind == 0 ? 0 : kind == 1 ? cq : cq + ck)) * kHeads;
    const int n = live ? min(kHeads, (kind == 0 ? a.Hq : a.Hkv) - h0) : 0;
    const Heads& src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const uint16_t* in = src.data + t * src.tok + h0 * src.head;
    const long long in_step = src.head;
    Part raw[kHeads][2];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
      if (i < n) {
        raw[i][0].load(in + i * in_step + at.o1);
        raw[i][1].load(in + i * in_step + at.o2);
      } else {
        raw[i][0] = raw[i][1] = Part{};
      }
    bool ok = live;
    if (!placed) {
      bad |= live;
      ok = false;
#pragma unroll
      for (int i = 0; i < kMaxAxes; ++i) pos.p[i] = 0;
    }
    uint16_t* out = a.q_out + ((long long)t * a.Hq + h0) * D;
    long long out_step = D;
    if (kCache) {
      const bool slot_ok = slot >= 0 && (slot >> a.page_shift) < a.pages;
      if (slot >= 0 && !slot_ok) bad |= live;
      if (kind) {
        const long long page = slot >> a.page_shift, row = slot & ((1 << a.page_shift) - 1);
        out = (kind == 1 ? a.k_cache : a.v_cache) + (((page * a.Hkv + h0) << a.page_shift) + row) * D;
        out_step = (long long)D << a.page_shift;
        ok = ok && slot_ok;
      }
    }
    const float* weight = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
    float c[2 * kPart], s[2 * kPart];
    coefficients(a, axes, at, which, pos, weight, c, s);
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      uint64_t v[kPart];
      turn<D, kF16, kInter>(raw[i], norms, weight != nullptr, a.eps, at.turns, c, s, v);
      Part y[2];
#pragma unroll
      for (int j = 0; j < kPart; ++j) y[j / (kPart / 2)].w[j % (kPart / 2)] = pack2<kF16>(lo(v[j]), hi(v[j]));
      if (!ok || i >= n) continue;
      uint16_t* dst = out + i * out_step;
      (kind == 2 ? raw[i][0] : y[0]).store(dst + at.o1);
      (kind == 2 ? raw[i][1] : y[1]).store(dst + at.o2);
    }
  }
  return bad;
}

}  // namespace
}  // namespace attn
}  // namespace moe
