// Attention weight of every key: what the rows of a call give to the keys of
// their sequences, added up over the rows and the G heads of a group,
//   weights[s, h, j] += sum_{t, g} exp(scale q[t, hG + g] . k[j, h] - lse[t, hG + g])
// over the rows t of sequence s that see key j.  lse comes from the attention
// call over the same rows, so that this needs one pass over the keys and no
// value is read.
//
// A warp takes 32 keys of one sequence and head and keeps them in registers as
// the B operand of mma.sync m16n8k16; the rows (token, head of the group) pass
// by in tiles of 16 as the A operand, both straight from global memory: a
// product's k index may stand for any element of D as long as it is the same one
// in both, so lane (g, q) of a fragment takes the contiguous elements q D/4 ..
// of row g, with 16-byte loads.  The exponentials are summed per key in
// registers, over the rows of a tile and from tile to tile; an entry belongs to
// one warp, which adds once: no atomics, the same bits every time.
//   The work of all sequences forms one line, a unit of 32 keys and a head
// weighing its row tiles and kUnitCost for its keys; the warps of the grid take
// equal ranges of it.
// Bound: single tokens HBM (2 D bytes a key and head), many rows the
// exponentials (one per row, head and key).
#include "attn.h"
#include "attn_ptx.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTiles = 4;             // of 8 keys: those of a unit
constexpr int kUnit = 8 * kTiles;
constexpr int kResident = 3;

template <bool kF16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kF16) mma_f16_16816(c, a[0], a[1], a[2], a[3], b0, b1);
  else mma_bf16_16816(c, a[0], a[1], a[2], a[3], b0, b1);
}

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
constexpr int kUnitCost = 2;          // a unit's keys, in row tiles
// Row tiles of a sequence's unit, its cost, and its units (of all heads)
__device__ __forceinline__ int tiles_of(const Seq& v, int G) { return (int)(((long long)v.n * G + 15) / 16); }
__device__ __forceinline__ long long line_of(const Seq& v, int G, int Hkv) {
  return v.n ? (long long)((v.len + kUnit - 1) / kUnit) * Hkv * (tiles_of(v, G) + kUnitCost) : 0;
}

template <int D, bool kF16>
__global__ void __launch_bounds__(kThreads, kResident) attn_weights_kernel(const WeightArgs a, const Report rep) {
  constexpr int kSteps = D / 16, kLoads = D / 32;      // 16-byte loads of a lane's part of a row
  __shared__ long long scan[kWarps], from[kWarps];
  __shared__ int from_seq[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, quad = lane & 3;
  const int G = a.Hq / a.Hkv;
  bool bad = false;
  // --- the line: every thread sums a run of sequences
  const int run = (a.n_seq + kThreads - 1) / kThreads;
  const int s0 = min(a.n_seq, (int)threadIdx.x * run), s1 = min(a.n_seq, s0 + run);
  if (threadIdx.x == 0) bad |= a.q_starts[0] != 0 || a.q_starts[a.n_seq] != a.T;
  long long mine = 0;
  for (int s = s0; s < s1; ++s) mine += line_of(seq_of(a, s, bad), G, a.Hkv);
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  if (lane == 0) from_seq[warp] = -1;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  // where each warp's range begins: found by the thread whose run it lies in
  const long long warps = (long long)gridDim.x * kWarps;
  const long long each = (total + warps - 1) / warps;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const long long at = ((long long)blockIdx.x * kWarps + w) * each;
    if (at < before || at >= before + mine) continue;
    long long p = before;
    for (int s = s0; s < s1; ++s) {
      const long long n = line_of(seq_of(a, s, bad), G, a.Hkv);
      if (at < p + n) {
        from_seq[w] = s;
        from[w] = p;
        break;
      }
      p += n;
    }
  }
  __syncthreads();
  const long long begin = ((long long)blockIdx.x * kWarps + warp) * each, end = begin + each;
  int s = from_seq[warp];
  if (s >= 0) {
    long long at = from[warp];                     // of the sequence
    Seq v = seq_of(a, s, bad);
    int tiles = tiles_of(v, G), units = (v.len + kUnit - 1) / kUnit;
    // a unit belongs to the warp whose range holds its first place
    long long u = (begin - at + tiles + kUnitCost - 1) / (tiles + kUnitCost);
    // the unit after, and its pages, while one is computed
    bool more = true;
    int pages[kTiles];
    auto fetch = [&]() {
      while (u >= (long long)units * a.Hkv) {      // to the next sequence with units
        if (++s >= a.n_seq) break;
        at += (long long)units * a.Hkv * (tiles + kUnitCost);
        v = seq_of(a, s, bad);
        tiles = tiles_of(v, G);
        units = v.n ? (v.len + kUnit - 1) / kUnit : 0;
        u = 0;
      }
      more = s < a.n_seq && at + u * (tiles + kUnitCost) < end;
      if (!more) return;
      const int k = (int)(u % units) * kUnit + gq;
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
        pages[i] = k + 8 * i < v.len ? a.page_table[(long long)s * a.table_pages + ((k + 8 * i) >> a.page_shift)] : 0;
    };
    fetch();
    uint32_t qf[2][kLoads][4];
    float off[2];
    int last[2];                                   // last key that a row sees
    int held = -1;                                 // the only row tile of this unit's sequence and head is in hand
#pragma unroll 1
    while (more) {
      const int seq = s, head = (int)(u / units), k0 = (int)(u - (long long)head * units) * kUnit, rowtiles = tiles;
      const Seq cur = v;
      // --- the keys: those past the end are not read
      uint32_t kf[kTiles][kLoads][4];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const int key = k0 + 8 * i + gq;
        int page = pages[i];
        if ((unsigned)page >= (unsigned)a.pages) bad = true, page = 0;
        const long long row =
            (((long long)page * a.Hkv + head) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
        const uint4* src = reinterpret_cast<const uint4*>(a.k_cache + row * D + quad * (D / 4));
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (key < cur.len) w = ldg_nc_v4(src + x);
          kf[i][x][0] = w.x, kf[i][x][1] = w.y, kf[i][x][2] = w.z, kf[i][x][3] = w.w;
        }
      }
      ++u;
      fetch();
      // --- the rows that see any of them
      const int shift = cur.len - cur.n;           // causal: token i sees the keys up to i + shift
      const int first = a.causal ? max(0, k0 - shift) : 0;
      const int rows = cur.n * G;
      float sum[kTiles][2];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) sum[i][0] = sum[i][1] = 0.f;
#pragma unroll 1
      for (int t = (int)((long long)first * G / 16); t < rowtiles; ++t) {
        if (rowtiles > 1 || held != seq * a.Hkv + head) {
          held = rowtiles > 1 ? -1 : seq * a.Hkv + head;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = 16 * t + 8 * x + gq;
            const bool live = r < rows;
            const int i = a.by_G.of(live ? r : 0), h = head * G + (live ? r : 0) - i * G;
            const uint16_t* src = a.q.data + (cur.q0 + i) * a.q.tok + h * a.q.head + quad * (D / 4);
            const float l = live ? a.lse[(long long)(cur.q0 + i) * a.Hq + h] : -INFINITY;
            // a row without keys, and one that is not there, give nothing
            off[x] = l == -INFINITY ? -INFINITY : -l * 1.4426950408889634f;
            last[x] = a.causal ? min(i + shift, cur.len - 1) : cur.len - 1;
#pragma unroll
            for (int y = 0; y < kLoads; ++y) {
              uint4 w = make_uint4(0, 0, 0, 0);
              if (live) w = *(reinterpret_cast<const uint4*>(src) + y);
              qf[x][y][0] = w.x, qf[x][y][1] = w.y, qf[x][y][2] = w.z, qf[x][y][3] = w.w;
            }
          }
        }
        const bool whole = __all_sync(0xffffffffu, last[0] >= k0 + kUnit - 1 && last[1] >= k0 + kUnit - 1);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            const uint32_t f[4] = {qf[0][k / 2][k % 2 * 2], qf[1][k / 2][k % 2 * 2], qf[0][k / 2][k % 2 * 2 + 1],
                                   qf[1][k / 2][k % 2 * 2 + 1]};
            mma<kF16>(c, f, kf[i][k / 2][k % 2 * 2], kf[i][k / 2][k % 2 * 2 + 1]);
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int x = y >> 1, key = k0 + 8 * i + 2 * quad + (y & 1);
            float e = ex2(fmaf(c[y], a.c, off[x]));
            if (off[x] == -INFINITY || (!whole && key > last[x])) e = 0.f;
            sum[i][y & 1] += e;
          }
        }
      }
      // --- over the eight rows of a tile that other lanes have; lane (gq, quad) adds key 8 (gq / 2) + 2 quad + gq % 2
      float add = 0.f;
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float e = sum[i][y];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) e += __shfl_xor_sync(0xffffffffu, e, d);
          if (gq == 2 * i + y) add = e;
        }
      const int key = k0 + 8 * (gq >> 1) + 2 * quad + (gq & 1);
      if (key < cur.len) {
        float* w = a.weights + ((long long)seq * a.Hkv + head) * a.capacity + key;
        *w += add;
      }
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) report(rep, blockIdx.x, any ? kStatusBounds : 0);
}

}  // namespace

cudaError_t launch_attn_weights(const WeightArgs& a, void* ws, int num_sms, cudaStream_t stream) {
  const int grid = num_sms * kResident;
  const Report rep{ws, 0, {grid, 0}};
  auto kern = a.D == 64 ? (a.f16 ? attn_weights_kernel<64, true> : attn_weights_kernel<64, false>)
                        : (a.f16 ? attn_weights_kernel<128, true> : attn_weights_kernel<128, false>);
  kern<<<grid, kThreads, 0, stream>>>(a, rep);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace moe
