// Attention with one warp per output row: the plain single-pass form.
//
// A warp owns (row t, head h), lanes split the head's D elements, and walks
// the visible keys with the running maximum m and sum l of the softmax:
//   s = scale q.k;  m' = max(m, s);  l = l e^{m-m'} + e^{s-m'};
//   o = o e^{m-m'} + e^{s-m'} v;     out = o / l,  lse = m + log l
#include "attn.h"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = 256;

template <bool kF16>
__device__ __forceinline__ float elem(const uint16_t* p) {
  if (kF16) {
    float f;
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(*p));
    return f;
  }
  return __uint_as_float((uint32_t)*p << 16);
}

template <int D, bool kF16>
__global__ void __launch_bounds__(kThreads) attn_rows_kernel(const AttnArgs a, const Report rep) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)a.T * a.Hq;
  bool bad = false;
  for (long long r = (long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; r < rows;
       r += (long long)gridDim.x * (kThreads / 32)) {
    const int t = (int)(r / a.Hq), h = (int)(r % a.Hq), hk = h / (a.Hq / a.Hkv);
    int s = t, q0 = t, q1 = t + 1;
    if (a.q_starts) {                      // last sequence that starts at or before t
      int lo = 0, hi = a.n_seq - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.q_starts[mid] <= t) lo = mid; else hi = mid - 1;
      }
      s = lo;
      q0 = a.q_starts[s];
      q1 = a.q_starts[s + 1];
      if (t < q0 || t >= q1) continue;
      if (q0 < 0 || q1 > a.T) { bad = true; continue; }
    }
    int k0 = 0, len;
    if (a.page_table) {
      len = a.kv_lens[s];
      if (len < 0 || len > ((long long)a.table_pages << a.page_shift)) { bad = true; continue; }
    } else {
      k0 = a.kv_starts[s];
      len = a.kv_starts[s + 1] - k0;
      if (k0 < 0 || len < 0 || k0 > a.Tk - len) { bad = true; continue; }
    }
    int seen = a.causal ? min(len, len - (q1 - q0) + (t - q0) + 1) : len;
    float q[N], o[N], m = -INFINITY, l = 0.f;
    for (int i = 0; i < N; ++i) {
      q[i] = elem<kF16>(a.q.data + t * a.q.tok + h * a.q.head + lane * N + i) * a.scale;
      o[i] = 0.f;
    }
    for (int j = -a.prefix_len; j < seen; ++j) {
      const uint16_t *kp, *vp;
      if (a.page_table) {
        const int jj = j < 0 ? j + a.prefix_len : j;
        const int* list = j < 0 ? a.prefix_table : a.page_table + (long long)s * a.table_pages;
        int page = list[jj >> a.page_shift];
        if ((unsigned)page >= (unsigned)a.pages) { bad = true; page = 0; }
        const long long at = ((((long long)page * a.Hkv + hk) << a.page_shift) + (jj & ((1 << a.page_shift) - 1))) * D;
        kp = a.k_cache + at;
        vp = a.v_cache + at;
      } else {
        kp = a.k.data + (k0 + j) * a.k.tok + hk * a.k.head;
        vp = a.v.data + (k0 + j) * a.v.tok + hk * a.v.head;
      }
      float x = 0.f;
      for (int i = 0; i < N; ++i) x = fmaf(q[i], elem<kF16>(kp + lane * N + i), x);
      for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      const float m2 = fmaxf(m, x), up = __expf(m - m2), p = __expf(x - m2);
      l = l * up + p;
      for (int i = 0; i < N; ++i) o[i] = o[i] * up + p * elem<kF16>(vp + lane * N + i);
      m = m2;
    }
    const float inv = l > 0.f ? 1.0f / l : 0.f;
    for (int i = 0; i < N; ++i) a.out[r * D + lane * N + i] = kF16 ? f2h(o[i] * inv) : f2bf(o[i] * inv);
    if (a.lse && lane == 0) a.lse[r] = l > 0.f ? m + logf(l) : -INFINITY;
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) report(rep, any ? kStatusBounds : 0);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs& a, const Report& shape, int num_sms, cudaStream_t stream) {
  const long long blocks = ((long long)a.T * a.Hq + kThreads / 32 - 1) / (kThreads / 32);
  const int grid = (int)(blocks < 8ll * num_sms ? blocks : 8ll * num_sms);
  Report rep = shape;
  rep.blocks[rep.set] = grid;
  auto kern = a.D == 64 ? (a.f16 ? attn_rows_kernel<64, true> : attn_rows_kernel<64, false>)
                        : (a.f16 ? attn_rows_kernel<128, true> : attn_rows_kernel<128, false>);
  kern<<<grid, kThreads, 0, stream>>>(a, rep);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace moe
