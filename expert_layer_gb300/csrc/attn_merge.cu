// Joins the parts of rows whose keys were split over blocks: with part i's
// result o_i and log2-sum lse_i,
//   out = sum_i w_i o_i / sum_i w_i,  w_i = 2^{lse_i - max lse},
//   lse = max lse + log2 sum_i w_i.
// A part without keys has lse_i = -inf; its o_i is not used.  The order of the
// parts is fixed, so the result does not change from run to run.
//
// Bound: latency (a row's parts are a few KB, just written).  A block takes a
// row, its four warps every fourth part each, with their loads in batches.
// Measured: 2048 rows of 16 parts (64 sequences behind a shared prefix) 4.5 us,
// 32 rows of 38 parts 5.
#include "attn.h"
#include "attn_ptx.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kBatch = 6;            // 4, 6, 8 with 19 parts a row: 41.2, 40.3, 41.3 us a call

struct MergeArgs {
  AttnArgs a;
  int splits;            // parts in row order: [splits, T * Hq]; 0: decode without a prefix
  DecodeParts p;
  int chunks;            // decode: units per key-value head
  int G, rows;           // heads of a key-value head; of a unit, at most 16
  Divisor by_rows, by_chunks, by_Hq, by_G;
  unsigned todo;         // rows to write
};

// Work: the rows, or, without parts in row order, the rows of the units that
// cross the decode kernel's blocks, at most one for each block.  (With 16 rows a
// unit whatever G, the blocks took two rounds: 64 sequences of 1466 keys, G = 8,
// 40.2 us against 39.0.)
template <int D, bool kF16, bool kPrefill>
__global__ void __launch_bounds__(kWarps * 32) attn_merge_kernel(const MergeArgs t) {
  constexpr int N = D / 32;            // elements per lane
  __shared__ float s_o[kWarps][D];
  __shared__ float2 s_ml[kWarps];
  const AttnArgs& a = t.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = t.G;
  const long long rows = (long long)a.T * a.Hq;
  // Rows of no sequence (reported by the kernel before) have no parts and stay
  // as they are.  Whether there are any is seen while that kernel runs; a call
  // with parts has few sequences (tc_splits).
  bool tidy = true;
  if (kPrefill) {
    for (int s = lane; s < a.n_seq; s += 32) tidy &= a.q_starts[s] <= a.q_starts[s + 1];
    tidy = __all_sync(0xffffffffu, tidy) && a.q_starts[0] == 0 && a.q_starts[a.n_seq] == a.T;
  }
  pdl_wait();   // programmatic dependent launch: the parts are complete
#pragma unroll 1
  for (unsigned i = blockIdx.x; i < t.todo; i += gridDim.x) {
    // blocks c0 .. c0 + own - 1 of the decode kernel hold the row's own keys
    int c0 = 0, own = 0, r = 0, parts = 0;
    long long row = i;
    bool ours = tidy;
    if (kPrefill && !tidy) {
      const int token = t.by_Hq.of((int)i);
      for (int s = lane; s < a.n_seq; s += 32) {
        const int q0 = a.q_starts[s], q1 = a.q_starts[s + 1];
        ours |= q0 >= 0 && q0 <= token && token < q1 && q1 <= a.T;
      }
      ours = __any_sync(0xffffffffu, ours);
    }
    if (!kPrefill && !t.splits) {
      c0 = t.by_rows.of((int)i);
      r = (int)i - c0 * t.rows;
      const int4 u = t.p.tail[c0];
      const int hk = t.by_chunks.of(u.y), h = (u.y - hk * t.chunks) * 16 + r;
      if (u.z == 0 || h >= G) continue;
      parts = own = u.z;
      row = (long long)u.x * a.Hq + hk * G + h;
    } else {
      parts = t.splits;
      if (!kPrefill) {
        const int b = t.by_Hq.of((int)i), h = (int)i - b * a.Hq, hk = t.by_G.of(h), g = h - hk * G;
        const int2 u = t.p.held[(b * a.Hkv + hk) * t.chunks + g / 16];
        own = u.x;
        c0 = u.y;
        r = g % 16;
        parts += own;
      }
    }
    float m = -INFINITY, sum = 0.f, acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.f;
#pragma unroll 1
    for (int i0 = warp; i0 < parts; i0 += kWarps * kBatch) {
      float lse[kBatch], o[kBatch][N];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kWarps;
        const float *po, *pl;
        if (i < t.splits || (t.splits && own == 1)) {      // the row's own part follows the prefix's
          const long long at = (long long)i * rows + row;
          po = t.p.tc_o + at * D;
          pl = t.p.tc_lse + at;
        } else {
          const int c = c0 + i - t.splits;
          const long long at = (2ll * c + (c == c0 ? 1 : 0)) * 16 + r;
          po = t.p.slot_o + at * D;
          pl = t.p.slot_lse + at;
        }
        lse[k] = i < parts ? *pl : -INFINITY;
#pragma unroll
        for (int j = 0; j < N; ++j) o[k][j] = i < parts ? po[lane * N + j] : 0.f;
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) top = fmaxf(top, lse[k]);
      const float zero = top == -INFINITY ? 0.f : top;    // parts that are all NaN have no maximum, and stay NaN
      const float f = ex2(m - zero);
      sum *= f;
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] *= f;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const bool none = lse[k] == -INFINITY;
        const float w = ex2(lse[k] - zero);
        sum += w;
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = fmaf(w, none ? 0.f : o[k][j], acc[j]);
      }
      m = top;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) s_o[warp][lane * N + j] = acc[j];
    if (lane == 0) s_ml[warp] = make_float2(m, sum);
    __syncthreads();
    const int x = threadIdx.x;
    if (x < D / 2 && ours) {
      float top = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w].x);
      if (top == -INFINITY) top = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(s_ml[w].x - top);
        l = fmaf(f, s_ml[w].y, l);
        o0 = fmaf(f, s_o[w][2 * x], o0);
        o1 = fmaf(f, s_o[w][2 * x + 1], o1);
      }
      const float inv = l > 0.f ? 1.0f / l : l;      // no keys: 0; NaN stays
      const uint32_t out = pack2<kF16>(o0 * inv, o1 * inv);
      const float lse = l == 0.f ? -INFINITY : (top + lg2(l)) * 0.693147180559945f;
      reinterpret_cast<uint32_t*>(a.out + row * D)[x] = out;
      if (a.lse && x == 0) a.lse[row] = lse;
    }
    __syncthreads();
  }
}

template <int D, bool kF16>
auto kernel_of(bool prefill) {
  return prefill ? attn_merge_kernel<D, kF16, true> : attn_merge_kernel<D, kF16, false>;
}

}  // namespace

cudaError_t launch_attn_merge(const AttnArgs& a, int splits, const DecodeParts& p, int decode_grid,
                              cudaStream_t stream) {
  MergeArgs t{};
  t.a = a;
  t.splits = splits;
  t.p = p;
  t.chunks = decode_chunks(a);
  t.G = a.Hq / a.Hkv;
  t.rows = t.G < 16 ? t.G : 16;
  t.by_rows.set(t.rows);
  t.by_chunks.set(t.chunks);
  t.by_Hq.set(a.Hq);
  t.by_G.set(t.G);
  t.todo = splits ? (unsigned)a.T * a.Hq : t.rows * decode_grid;
  const bool rows = decode_grid == 0;
  auto kern = a.D == 64 ? (a.f16 ? kernel_of<64, true>(rows) : kernel_of<64, false>(rows))
                        : (a.f16 ? kernel_of<128, true>(rows) : kernel_of<128, false>(rows));
  return launch_pdl(kern, dim3(t.todo < 2560 ? t.todo : 2560), dim3(kWarps * 32), 0, stream, t);
}

}  // namespace attn
}  // namespace moe
