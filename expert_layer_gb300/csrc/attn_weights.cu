// Attention weight of every key: what the rows of a call give to the keys of
// their sequences, added up over the rows and the G heads of a group,
//   weights[s, h, j] += sum_{t, g} exp(scale q[t, hG + g] . k[j, h] - lse[t, hG + g])
// over the rows t of sequence s that see key j.  lse comes from the attention
// call over the same rows, so that this needs one pass over the keys and no
// value is read.
//
// A warp takes 16 keys (D = 64: 32) of one sequence and head and keeps them in
// registers as the B operand of mma.sync m16n8k16; the rows (token, head of the
// group) pass by in tiles of 16 as the A operand, both straight from global
// memory: a product's k index may stand for any element of D as long as it is
// the same one in both, so lane (g, q) of a fragment takes the contiguous
// elements q D/4 .. of row g, with 16-byte loads.  The exponentials are summed
// per key in registers, over the rows of a tile and from tile to tile; an entry
// belongs to one warp, which adds once: no atomics, the same bits every time.
//   The work of all sequences forms one line, a unit of those keys and a head
// weighing its row tiles and kUnitCost for its keys; the warps of the grid take
// equal ranges of it.  Keys and entries are loaded a unit ahead, page ids two
// (32 keys at D = 128 with two blocks to an SM 17.6 us in place of 17.4; an entry
// read where it is written cost a warp its latency for every unit, 20.4).
// Calls with more rows go to the tensor cores (attn_weights_tc.cu): 16 sequences
// of 4000 keys, 4 heads of 128, with 8, 16, 24, 64 rows each here 17.8, 18.2,
// 25.6, 37.2 us, there 17.7, 17.8, 17.8, 20.8; 8 heads of 64 with 16 rows 18.6 and
// 28.2, one with 32 9.5 and 9.4.
// Bound: HBM (2 D bytes a key and head), of which 64 rows over 57 MB of keys read
// 3.3 TB/s in 17.4 us; 5.5 us are the start: a launch, lengths, page ids, keys.
#include "attn.h"
#include "attn_ptx.cuh"
#include "weights_line.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
template <int D>
constexpr int kTiles = D == 128 ? 2 : 4;      // of 8 keys: those of a unit
template <int D>
constexpr int kUnit = 8 * kTiles<D>;
constexpr int kResident = 3;
constexpr int kTcRows = 16;           // rows of a sequence and head, on average, above which the tensor cores take a call

template <bool kF16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kF16) mma_f16_16816(c, a[0], a[1], a[2], a[3], b0, b1);
  else mma_bf16_16816(c, a[0], a[1], a[2], a[3], b0, b1);
}

constexpr int kUnitCost = 2;          // a unit's keys, in row tiles
// Row tiles of a sequence's unit, its cost, and its units (of all heads)
__device__ __forceinline__ int tiles_of(const Seq& v, int G) { return (int)(((long long)v.n * G + 15) / 16); }
template <int D>
__device__ __forceinline__ long long line_of(const Seq& v, int G, int Hkv) {
  return v.n ? (long long)((v.len + kUnit<D> - 1) / kUnit<D>) * Hkv * (tiles_of(v, G) + kUnitCost) : 0;
}

template <int D, bool kF16>
__global__ void __launch_bounds__(kThreads, kResident) attn_weights_kernel(const WeightArgs a, const Report rep) {
  constexpr int kSteps = D / 16, kLoads = D / 32;      // 16-byte loads of a lane's part of a row
  constexpr int kTiles = attn::kTiles<D>, kUnit = attn::kUnit<D>;
  __shared__ LineStart<kThreads> start;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, quad = lane & 3;
  const int G = a.Hq / a.Hkv;
  bool bad = false;
  find_start(a, start, kWarps, [&](const Seq& v) { return line_of<D>(v, G, a.Hkv); }, bad);
  const long long range = (long long)blockIdx.x * kWarps + warp, begin = start.begin(range), end = start.begin(range + 1);
  int s = start.seq[warp];
  if (s >= 0) {
    long long at = start.at[warp];                 // of the sequence
    Seq v = seq_of(a, s, bad);
    int tiles = tiles_of(v, G), units = (v.len + kUnit - 1) / kUnit;
    // a unit belongs to the warp whose range holds its first place
    const long long u = (begin - at + tiles + kUnitCost - 1) / (tiles + kUnitCost);
    int head = units ? (int)(u / units) : a.Hkv, index = (int)(u - (long long)head * units);
    at += u * (tiles + kUnitCost);                 // place of the unit
    // Three units under way: one is computed while the keys of the next are
    // loaded and the page ids of the one after.
    struct Keys {
      int seq, head, k0, rowtiles;                 // seq -1: no unit
      Seq v;
      float* to;
      float held;
      uint32_t f[kTiles][kLoads][4];
    };
    bool more = true;
    int pages[kTiles];
    auto fetch = [&]() {
      while (head >= a.Hkv) {                      // to the next sequence with units
        if (++s >= a.n_seq) break;
        v = seq_of(a, s, bad);
        tiles = tiles_of(v, G);
        units = v.n ? (v.len + kUnit - 1) / kUnit : 0;
        head = units ? 0 : a.Hkv;
        index = 0;
      }
      more = s < a.n_seq && at < end;
      if (!more) return;
      const int k = index * kUnit + gq;
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
        pages[i] = k + 8 * i < v.len ? a.page_table[(long long)s * a.table_pages + ((k + 8 * i) >> a.page_shift)] : 0;
    };
    auto load = [&](Keys& w) {                     // those past the end are not read
      w.seq = -1;
      if (!more) return;
      w.seq = s, w.head = head, w.k0 = index * kUnit, w.rowtiles = tiles;
      w.v = v;
      // lane (gq, quad) adds to key 8 (gq / 2) + 2 quad + gq % 2: what it holds is on its way meanwhile
      const int key = w.k0 + 8 * (gq >> 1) + 2 * quad + (gq & 1);
      w.to = gq < 2 * kTiles && key < v.len ? a.weights + ((long long)s * a.Hkv + head) * a.capacity + key : nullptr;
      w.held = w.to ? *w.to : 0.f;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const int key = w.k0 + 8 * i + gq;
        int page = pages[i];
        if ((unsigned)page >= (unsigned)a.pages) bad = true, page = 0;
        const long long row =
            (((long long)page * a.Hkv + w.head) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
        const uint4* src = reinterpret_cast<const uint4*>(a.k_cache + row * D + quad * (D / 4));
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
          uint4 k = make_uint4(0, 0, 0, 0);
          if (key < v.len) k = ldg_nc_v4(src + x);
          w.f[i][x][0] = k.x, w.f[i][x][1] = k.y, w.f[i][x][2] = k.z, w.f[i][x][3] = k.w;
        }
      }
      at += tiles + kUnitCost;
      if (++index == units) index = 0, ++head;
      fetch();
    };
    uint32_t qf[2][kLoads][4];
    float off[2];
    int last[2];                                   // last key that a row sees
    int held = -1;                                 // the only row tile of this sequence and head is in hand
    auto compute = [&](const Keys& w) {
      const int seq = w.seq, head = w.head, k0 = w.k0, rowtiles = w.rowtiles;
      const Seq& cur = w.v;
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
            mma<kF16>(c, f, w.f[i][k / 2][k % 2 * 2], w.f[i][k / 2][k % 2 * 2 + 1]);
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
      // --- over the eight rows of a tile that other lanes have
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
      if (w.to) *w.to = w.held + add;
    };
    Keys ka, kb;
    fetch();
    load(ka);
#pragma unroll 1
    while (ka.seq >= 0) {
      load(kb);
      compute(ka);
      if (kb.seq < 0) break;
      load(ka);
      compute(kb);
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) report(rep, blockIdx.x, any ? kStatusBounds : 0);
}

}  // namespace

cudaError_t launch_attn_weights(const WeightArgs& a, void* ws, int num_sms, cudaStream_t stream) {
  if ((long long)a.T * (a.Hq / a.Hkv) > (long long)kTcRows * a.n_seq)
    return launch_attn_weights_tc(a, ws, num_sms, stream);
  const int grid = num_sms * kResident;
  const Report rep{ws, 0, {grid, 0}};
  auto kern = a.D == 64 ? (a.f16 ? attn_weights_kernel<64, true> : attn_weights_kernel<64, false>)
                        : (a.f16 ? attn_weights_kernel<128, true> : attn_weights_kernel<128, false>);
  kern<<<grid, kThreads, 0, stream>>>(a, rep);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace moe
