// Attention of single tokens over the paged cache.
//
// A unit is one sequence's token on one key-value head: its G query heads
// (at most 16; larger groups make several units) share every key and value
// that is read.  The keys of all units form one line of 16-key slices (a
// slice lies within a page), a unit's slices after one place that stands for
// the unit's own cost, cut into equal ranges for the blocks, so that lengths as
// different as 1 and 100,000 load the GPU evenly; a unit that spans blocks
// leaves one part per block and the merge kernel joins them.
//
// Bound: HBM (4 D bytes per key and key-value head against 4 G D flops).  A
// block's range is cut once more over its eight warps, each of which works
// alone on consecutive slices with its softmax state, m, l and O in
// registers, and keeps a ring of slices filled by TMA, across units: no
// barrier until the block's end.  A unit that lies within a warp's range is
// finished there; what a warp holds of a unit that crosses its range goes to
// shared memory, where the block joins it at its end.
//   S = Q K^T, O += P V   mma.sync m16n8k16, rows = heads (8 or 16 of 16)
// mma.sync rather than tcgen05: a unit has 8 or 16 rows of the 128 that the
// latter multiplies, and the kernel waits for HBM in any case (issue slots 20%
// used, mma pipe 14%).
// P is rounded to the element type for the second product, l sums it before
// that: error against 64 bits 1.7e-3 where weights in 32 bits leave 1.5e-3 (64
// sequences of 1 to 8192 keys, bf16; attn_tc.cu says more).
// Measured (32 query and 4 key-value heads of 128, bf16): 128 sequences of 4096
// keys 167 us = 6.4 TB/s, 95% of a copy's rate; one of 131,001 keys 49.9 us, of
// which it streams 38 at 6.9 TB/s; 64 of 1 to 8192 keys 26.8; 1024 of 90 keys
// 46.9; 8 of 400 keys 9.5, the keys themselves 1 (the rest is start, join and
// merge).
#include "attn.h"
#include "attn_ptx.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kSlice = 16;          // keys
constexpr int kWindow = kThreads;   // sequences whose lengths a block keeps in shared memory
constexpr float kLag = 8.0f;        // log2 of how far the maximum in use may lag

template <int D, bool kWide>
struct Shape {
  static constexpr int kRows = kWide ? 16 : 8;                     // heads of a unit
  static constexpr int kHalves = D / 64;
  static constexpr int kGroup = kHalves * 1024;                    // 8 keys: kHalves swizzle atoms
  static constexpr int kTileBytes = 2 * kGroup;                    // K or V of a slice
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = D == 64 ? 5 : kWide ? 2 : 3;      // slices in flight per warp
  static constexpr int kRing = kStages * kStageBytes;              // of one warp
  static constexpr int kPart = kRows * D * 4;                      // O of one unit
  static_assert(kPart <= kRing, "a warp's last part takes the place of its ring");
  static constexpr int kFirst = kWarps * kRing;                    // O of the warps' first parts
  static constexpr int kStats = kFirst + kWarps * kPart;           // m and l of the rows, two parts per warp
  static constexpr int kOpen = kStats + kWarps * 2 * kRows * 8;       // the units that the parts belong to
  static constexpr int kBars = kOpen + kWarps * 2 * 16;
  static constexpr int kLens = kBars + kWarps * kStages * 8;
  static constexpr int kScan = kLens + kWindow * 4;
  static constexpr size_t kSmem = kScan + 128;
};
static_assert(Shape<128, false>::kSmem <= 232448 && Shape<128, true>::kSmem <= 232448, "227 KB a block");

// The units of a range: a cursor over (sequence, unit of the sequence),
// empty sequences left out.  `pos` is the unit's place on the line; its slices
// come kUnitCost later.
struct Cursor {
  int b, u, len, slices, pos;
};
// A unit that a warp holds a part of (b < 0: none)
struct Open {
  int b, u, slices, pos;
};

struct DecodeArgs {
  AttnArgs a;
  float c;              // |scale| log2 e, > 0
  uint32_t flip;        // sign bits of two elements when the scale is negative
  int G;                // Hq / Hkv
  int chunks;           // units per key-value head
  int few, head;        // of Line
  int arrivals;         // that a stage's barrier waits for: 1, or one too many
  DecodeParts p;
};

template <bool kF16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if (kF16) mma_f16_16816(c, a0, a1, a2, a3, b0, b1);
  else mma_bf16_16816(c, a0, a1, a2, a3, b0, b1);
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ int seq_len(const AttnArgs& a, int b) {
  const int n = a.kv_lens[b];
  return n < 0 || n > ((long long)a.table_pages << a.page_shift) ? 0 : n;
}
__device__ __forceinline__ int slices_of(int len) { return (len + kSlice - 1) / kSlice; }
// Places that a unit of `len` keys takes on the line
__device__ __forceinline__ int unit_weight(int len) { return len > 0 ? slices_of(len) + kUnitCost : 0; }

// Lengths of the sequences from b0 on, the first kWindow of them in shared memory
struct Lens {
  const AttnArgs* a;
  const int* window;
  int b0;
  __device__ __forceinline__ int operator()(int b) const {
    return b - b0 < kWindow ? window[b - b0] : seq_len(*a, b);
  }
};

// To the next unit that has slices (or past the last sequence).
__device__ __forceinline__ void advance(const Lens& lens, Cursor& c, int units) {
  c.pos += c.slices + kUnitCost;
  if (++c.u < units) return;
  c.u = 0;
  c.slices = 0;
  while (++c.b < lens.a->n_seq) {
    c.len = lens(c.b);
    c.slices = slices_of(c.len);
    if (c.slices) break;
  }
}

template <int D, bool kF16, bool kWide>
__global__ void __launch_bounds__(kThreads, 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const DecodeArgs t, const Report rep) {
  using S = Shape<D, kWide>;
  constexpr int kRowSets = kWide ? 2 : 1;            // rows g and (wide) g + 8 of a thread
  constexpr int kStages = S::kStages;
  extern __shared__ __align__(1024) unsigned char smem[];      // swizzle atoms of 1 KB
  float2* stats = reinterpret_cast<float2*>(smem + S::kStats);         // [warp][part][row]: m, l
  Open* open = reinterpret_cast<Open*>(smem + S::kOpen);               // [warp][part]
  int* window = reinterpret_cast<int*>(smem + S::kLens);
  int* scan = reinterpret_cast<int*>(smem + S::kScan);     // [8] warp sums, then the start
  const AttnArgs& a = t.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = t.G, units = a.Hkv * t.chunks;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars) + warp * kStages;
  unsigned char* ring = smem + warp * S::kRing;
  bool bad = false, late = false;
  pdl_trigger();     // the merge kernel may become resident; it waits for this grid's end
  if (threadIdx.x == 0) {
    prefetch_map(&tmK);
    prefetch_map(&tmV);
  }

  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&bars[i], t.arrivals);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    open[2 * warp].b = open[2 * warp + 1].b = -1;
  }

  // --- the line of slices: every thread sums a run of sequences
  const int run = (a.n_seq + kThreads - 1) / kThreads;
  const int s0 = min(a.n_seq, (int)threadIdx.x * run), s1 = min(a.n_seq, s0 + run);
  int mine = 0;
  for (int s = s0; s < s1; ++s) {
    const int n = a.kv_lens[s];
    const bool fits = n >= 0 && n <= ((long long)a.table_pages << a.page_shift);
    if (blockIdx.x == 0 && !fits) bad = true;
    mine += unit_weight(fits ? n : 0) * units;
    if (run == 1) window[s] = fits ? n : 0;
  }
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  before += incl - mine;
  const Line line(total, gridDim.x, t.few, t.head);
  const int start = line.at(blockIdx.x * kWarps), end = line.at((blockIdx.x + 1) * kWarps);
  const bool work = (int)blockIdx.x < line.blocks && start < end;
  if (work && start >= before && start < before + mine) {
    int at = before;
    for (int s = s0; s < s1; ++s) {
      const int n = unit_weight(run == 1 ? window[s] : seq_len(a, s)) * units;
      if (start < at + n) {
        scan[kWarps] = s;
        scan[kWarps + 1] = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  Lens lens{&a, window, 0};
  if (work && run > 1) {
    lens.b0 = scan[kWarps];
    const int s = lens.b0 + threadIdx.x;
    window[threadIdx.x] = s < a.n_seq ? seq_len(a, s) : 0;
    __syncthreads();
  }

  // --- this warp's range
  const int ws = line.at(blockIdx.x * kWarps + warp), we = line.at(blockIdx.x * kWarps + warp + 1);
  if (work && ws < we) {
    Cursor cur;
    cur.b = scan[kWarps];
    cur.pos = scan[kWarps + 1];
    while (true) {                               // the sequence that ws lies in
      cur.len = lens(cur.b);
      cur.slices = slices_of(cur.len);
      const int n = unit_weight(cur.len) * units;
      if (ws < cur.pos + n) break;
      cur.pos += n;
      ++cur.b;
    }
    cur.u = (ws - cur.pos) / (cur.slices + kUnitCost);
    cur.pos += cur.u * (cur.slices + kUnitCost);

    // --- loads: the same walk, kStages slices ahead
    Cursor ld = cur;
    int ld_slice = max(0, ws - ld.pos - kUnitCost);
    uint32_t issued = 0;
    int page = 0;
    bool more;
    // the page id of slice `ld_slice` of ld, one slice before its load
    auto fetch = [&]() {
      if (ld_slice == ld.slices) {
        advance(lens, ld, units);
        ld_slice = 0;
      }
      more = ld.pos + kUnitCost + ld_slice < we;
      if (more) page = a.page_table[(long long)ld.b * a.table_pages + ((ld_slice * kSlice) >> a.page_shift)];
    };
    fetch();
    auto issue = [&]() {
      if (!more) return;
      if (lane == 0) {
        if ((unsigned)page >= (unsigned)a.pages) {
          bad = true;
          page = 0;
        }
        const int st = issued % kStages, row = (ld_slice * kSlice) & ((1 << a.page_shift) - 1);
        const int hk = t.chunks == 1 ? ld.u : ld.u / t.chunks;
        unsigned char* dst = ring + st * S::kStageBytes;
        mbar_expect_tx(&bars[st], S::kStageBytes);
        tma_load_5d(dst, &tmK, 0, 0, 0, row / 8, page * a.Hkv + hk, &bars[st]);
        tma_load_5d(dst + S::kTileBytes, &tmV, 0, 0, 0, row / 8, page * a.Hkv + hk, &bars[st]);
      }
      ++issued;
      ++ld_slice;
      fetch();
    };
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) issue();

    // ldmatrix source of this lane: K: 8x8 matrices (keys 0-7 | 8-15) x (d 0-7 | 8-15),
    // V transposed: the same with keys fastest; rows are swizzled by key % 8
    const int k_row = (lane & 7) + ((lane & 16) >> 1), k_col = (lane >> 3) & 1;
    const int v_row = (lane & 7) + (lane & 8), v_col = lane >> 4;
    const int k_at = (k_row >> 3) * S::kGroup + (k_row & 7) * 128, v_at = (v_row >> 3) * S::kGroup + (v_row & 7) * 128;
    const int quad = lane & 3, gq = lane >> 2;
    uint32_t used = 0;
    auto load_q = [&](const Cursor& c, uint32_t (&q)[D / 16][2 * kRowSets]) {
      const int hk = t.chunks == 1 ? c.u : c.u / t.chunks;
      const int h0 = hk * G + (c.u - hk * t.chunks) * 16, rows = min(16, hk * G + G - h0);
      const uint16_t* src = a.q.data + (long long)c.b * a.q.tok;
#pragma unroll
      for (int rs = 0; rs < kRowSets; ++rs) {
        const int r = gq + 8 * rs;
        const uint16_t* p = src + (long long)(h0 + (r < rows ? r : 0)) * a.q.head + 2 * quad;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          q[kk][rs] = r < rows ? *reinterpret_cast<const uint32_t*>(p + kk * 16) ^ t.flip : 0u;
          q[kk][kRowSets + rs] = r < rows ? *reinterpret_cast<const uint32_t*>(p + kk * 16 + 8) ^ t.flip : 0u;
        }
      }
    };
    uint32_t q[D / 16][2 * kRowSets];
    load_q(cur, q);

    while (cur.pos < we) {
      const int first = max(0, ws - cur.pos - kUnitCost), last = min(cur.slices, we - cur.pos - kUnitCost);
      Cursor nxt = cur;
      advance(lens, nxt, units);
      uint32_t qn[D / 16][2 * kRowSets];             // the next unit's, under way meanwhile
      if (!kWide && nxt.pos < we) load_q(nxt, qn);
      float o[D / 8][4];
      float m[kRowSets], l[kRowSets];
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
#pragma unroll
      for (int rs = 0; rs < kRowSets; ++rs) m[rs] = -INFINITY, l[rs] = 0.f;

#pragma unroll 1
      for (int s = first; s < last; ++s) {
        const int st = used % kStages;
        // after a timeout nothing more is loaded: a stage whose load has not
        // landed must not be loaded again, nor its barrier be armed again
        if (!late && !warp_spin(&bars[st], (used / kStages) & 1)) late = true, more = false;
        const uint32_t kb = smem_u32(ring + st * S::kStageBytes), vb = kb + S::kTileBytes;
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t r[4];
          const int chunk = (kk & 3) * 2 + k_col;
          ldsm4(kb + (kk >> 2) * 1024 + k_at + ((chunk ^ (k_row & 7)) << 4), r);
          const uint32_t a1 = kWide ? q[kk][kRowSets - 1] : 0u, a3 = kWide ? q[kk][2 * kRowSets - 1] : 0u;
          mma<kF16>(sc[0], q[kk][0], a1, q[kk][kRowSets], a3, r[0], r[1]);
          mma<kF16>(sc[1], q[kk][0], a1, q[kk][kRowSets], a3, r[2], r[3]);
        }
        // keys of this thread: 2 quad + {0, 1} of each half of the slice
        const int valid = cur.len - s * kSlice;
        if (valid < kSlice) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (8 * h + 2 * quad + (j & 1) >= valid) sc[h][j] = -INFINITY;
        }
        uint32_t p[4] = {0u, 0u, 0u, 0u};
        bool up = false;
        float top[kRowSets];
#pragma unroll
        for (int rs = 0; rs < kRowSets; ++rs) {
          float x = fmaxf(fmaxf(sc[0][2 * rs], sc[0][2 * rs + 1]), fmaxf(sc[1][2 * rs], sc[1][2 * rs + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          top[rs] = x * t.c;
          up |= top[rs] > m[rs] + kLag;
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int rs = 0; rs < kRowSets; ++rs) {
            const bool g = top[rs] > m[rs] + kLag;
            const float f = g ? ex2(m[rs] - top[rs]) : 1.0f;
            if (g) m[rs] = top[rs];
            l[rs] *= f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              o[i][2 * rs] *= f;
              o[i][2 * rs + 1] *= f;
            }
          }
        }
#pragma unroll
        for (int rs = 0; rs < kRowSets; ++rs) {
          const float off = m[rs] == -INFINITY ? 0.f : m[rs];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p0 = ex2(fmaf(sc[h][2 * rs], t.c, -off)), p1 = ex2(fmaf(sc[h][2 * rs + 1], t.c, -off));
            l[rs] += p0 + p1;
            p[2 * h + rs] = pack2<kF16>(p0, p1);
          }
        }
        // values past the end may be anything: a weight of 0 does not silence NaN
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (valid < kSlice) {
          const int k0 = 2 * quad;
          keep0 = (k0 < valid ? 0xffffu : 0u) | (k0 + 1 < valid ? 0xffff0000u : 0u);
          keep1 = (k0 + 8 < valid ? 0xffffu : 0u) | (k0 + 9 < valid ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t r[4];
          const int chunk = (i & 3) * 2 + v_col;
          ldsm4_t(vb + (i >> 2) * 1024 + v_at + ((chunk ^ (v_row & 7)) << 4), r);
          mma<kF16>(o[2 * i], p[0], p[1], p[2], p[3], r[0] & keep0, r[1] & keep1);
          mma<kF16>(o[2 * i + 1], p[0], p[1], p[2], p[3], r[2] & keep0, r[3] & keep1);
        }
        __syncwarp();            // every lane has read the stage
        ++used;
        issue();
      }

      // --- the end of this warp's part of the unit
#pragma unroll
      for (int rs = 0; rs < kRowSets; ++rs) {
        l[rs] += __shfl_xor_sync(0xffffffffu, l[rs], 1);
        l[rs] += __shfl_xor_sync(0xffffffffu, l[rs], 2);
      }
      if (last <= first) {
        // none of its slices: the range ends before them
      } else if (first == 0 && last == cur.slices) {
        const int hk = t.chunks == 1 ? cur.u : cur.u / t.chunks;
        const int h0 = hk * G + (cur.u - hk * t.chunks) * 16, rows = min(16, hk * G + G - h0);
#pragma unroll
        for (int rs = 0; rs < kRowSets; ++rs) {
          const int r = gq + 8 * rs;
          if (r >= rows) continue;
          const long long row = (long long)cur.b * a.Hq + h0 + r;
          // (every logit -inf: a weight of 0 and a log-sum of -inf, as without keys)
          const float inv = l[rs] > 0.f ? 1.0f / l[rs] : l[rs], lse = m[rs] + lg2(l[rs]);
          if (t.p.row_o) {
            if (lane == 0 && rs == 0) t.p.held[cur.b * units + cur.u] = make_int2(1, 0);
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              *reinterpret_cast<float2*>(t.p.row_o + row * D + 8 * i + 2 * quad) =
                  make_float2(o[i][2 * rs] * inv, o[i][2 * rs + 1] * inv);
            if (quad == 0) t.p.row_lse[row] = lse;
          } else {
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              *reinterpret_cast<uint32_t*>(a.out + row * D + 8 * i + 2 * quad) =
                  pack2<kF16>(o[i][2 * rs] * inv, o[i][2 * rs + 1] * inv);
            if (a.lse && quad == 0) a.lse[row] = lse * 0.693147180559945f;
          }
        }
      } else {
        // part 0: the unit began before this warp's range; part 1: it goes on
        // after it (every load of the ring has been consumed by then)
        const int part = first > 0 ? 0 : 1;
        float* dst = reinterpret_cast<float*>(part ? ring : smem + S::kFirst + warp * S::kPart);
#pragma unroll
        for (int rs = 0; rs < kRowSets; ++rs) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2*>(dst + (gq + 8 * rs) * D + 8 * i + 2 * quad) =
                make_float2(o[i][2 * rs], o[i][2 * rs + 1]);
          if (quad == 0) stats[(2 * warp + part) * S::kRows + gq + 8 * rs] = make_float2(m[rs], l[rs]);
        }
        if (lane == 0) open[2 * warp + part] = Open{cur.b, cur.u, cur.slices, cur.pos};
      }
      cur = nxt;
      if (kWide) {
        if (cur.pos < we) load_q(cur, q);
      } else {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int j = 0; j < 2 * kRowSets; ++j) q[kk][j] = qn[kk][j];
      }
    }
    // after a timeout: the loads already issued land before the block exits
    if (late && lane == 0)
      for (uint32_t i = issued > (uint32_t)kStages ? issued - kStages : 0; i < issued; ++i)
        spin_wait(&bars[i % kStages], (i / kStages) & 1);
  }
  __syncthreads();

  // --- rows without keys (with a prefix the merge kernel writes every row)
  for (int s = blockIdx.x; s < a.n_seq; s += gridDim.x)
    if ((run == 1 ? window[s] : seq_len(a, s)) == 0) {
      if (t.p.row_o) {
        for (int i = threadIdx.x; i < units; i += kThreads) t.p.held[s * units + i] = make_int2(0, 0);
      } else {
        for (int i = threadIdx.x; i < a.Hq * (D / 8); i += kThreads)
          reinterpret_cast<uint4*>(a.out + (long long)s * a.Hq * D)[i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
          for (int i = threadIdx.x; i < a.Hq; i += kThreads) a.lse[(long long)s * a.Hq + i] = -INFINITY;
      }
    }

  // --- join the warps' parts of units that cross their ranges: row r is
  // out = sum_w 2^{m_w - M} O_w / sum_w 2^{m_w - M} l_w.  The parts of a unit
  // follow one another in (warp, part) order.
  int4 tail = make_int4(0, 0, 0, 0);             // the unit that goes on in the next block
#pragma unroll 1
  for (int e = 0; e < 2 * kWarps; e = e == 0 ? 1 : e + 2) {      // part 0 of the first warp, part 1 of every warp
    const Open op = open[e];
    if (op.b < 0) continue;
    const int w0 = e >> 1;
    const Open other = open[2 * (lane & (kWarps - 1))];          // part 0 of the warps after it
    const int parts = 1 + __popc(__ballot_sync(0xffffffffu, lane < kWarps && lane > w0 && other.b == op.b &&
                                                                other.u == op.u));
    const int begin = op.pos + kUnitCost;
    const bool whole = begin >= start && begin + op.slices <= end;
    const int slot = 2 * blockIdx.x + (begin < start ? 0 : 1);
    if (begin >= start && !whole)
      tail = make_int4(op.b, op.u, line.block_of(begin + op.slices - 1) - (int)blockIdx.x + 1, 0);
    if (t.p.row_o && threadIdx.x == 0 && begin >= start)
      t.p.held[op.b * units + op.u] = whole ? make_int2(1, 0) : make_int2(tail.z, (int)blockIdx.x);
    const int hk = t.chunks == 1 ? op.u : op.u / t.chunks;
    const int h0 = hk * G + (op.u - hk * t.chunks) * 16, rows = min(16, hk * G + G - h0);
    for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      float2 ml[kWarps];
      float4 x[kWarps];
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < parts) {
          const int p = k == 0 ? e : 2 * (w0 + k);
          const unsigned char* at = p & 1 ? smem + (p >> 1) * S::kRing : smem + S::kFirst + (p >> 1) * S::kPart;
          ml[k] = stats[p * S::kRows + r];
          x[k] = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(at) + r * D + d);
        }
        M = fmaxf(M, ml[k].x);
      }
      float sum = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float w = M == -INFINITY ? 0.f : ex2(ml[k].x - M);
        sum = fmaf(w, ml[k].y, sum);
        v.x = fmaf(w, x[k].x, v.x);
        v.y = fmaf(w, x[k].y, v.y);
        v.z = fmaf(w, x[k].z, v.z);
        v.w = fmaf(w, x[k].w, v.w);
      }
      const float inv = sum > 0.f ? 1.0f / sum : sum;        // 0 stays 0, NaN stays NaN
      v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
      const float lse = M + lg2(sum);
      const long long row = (long long)op.b * a.Hq + h0 + r;
      if (whole && !t.p.row_o) {
        uint2 w;
        w.x = pack2<kF16>(v.x, v.y);
        w.y = pack2<kF16>(v.z, v.w);
        *reinterpret_cast<uint2*>(a.out + row * D + d) = w;
        if (a.lse && d == 0) a.lse[row] = lse * 0.693147180559945f;
      } else {
        const long long at = whole ? row : (long long)slot * 16 + r;
        *reinterpret_cast<float4*>((whole ? t.p.row_o : t.p.slot_o) + at * D + d) = v;
        if (d == 0) (whole ? t.p.row_lse : t.p.slot_lse)[at] = lse;
      }
    }
  }
  const int any_bad = __syncthreads_or(bad), any_late = __syncthreads_or(late);
  if (threadIdx.x == 0) t.p.tail[blockIdx.x] = tail;
  if (threadIdx.x == 0) report(rep, blockIdx.x, (any_bad ? kStatusBounds : 0) | (any_late ? kStatusTimeout : 0));
  // launched beside the prefix's kernel: this grid ends after it, so that the
  // merge kernel, which waits for this one, finds the parts of both (one block
  // waits; the others leave their SMs to blocks that have not started)
  if (blockIdx.x == 0) pdl_wait();
}

template <int D, bool kF16, bool kWide>
cudaError_t launch(const DecodeArgs& t, const CUtensorMap& k, const CUtensorMap& v, const Report& rep, bool beside,
                   int grid, cudaStream_t stream) {
  auto kern = attn_decode_kernel<D, kF16, kWide>;
  constexpr size_t smem = Shape<D, kWide>::kSmem;
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  if (beside) return launch_pdl(kern, dim3(grid), dim3(kThreads), smem, stream, k, v, t, rep);
  kern<<<grid, kThreads, smem, stream>>>(k, v, t, rep);
  return cudaGetLastError();
}

}  // namespace

// beside: the kernel before this one on the stream is the prefix's, on which
// nothing here depends
cudaError_t launch_attn_decode(const AttnArgs& a, const Beside& beside, const DecodeParts& p, const Report& shape,
                               int num_sms, cudaStream_t stream) {
  DecodeArgs t{};
  t.a = a;
  t.c = (a.scale < 0 ? -a.scale : a.scale) * 1.4426950408889634f;
  if (t.c < 1.2e-38f) t.c = 1.2e-38f;      // a masked logit of -inf stays one
  t.flip = a.scale < 0 ? 0x80008000u : 0u;
  const int G = a.Hq / a.Hkv;
  t.G = G;
  t.chunks = decode_chunks(a);
  t.few = beside.few;
  t.head = beside.head;
  t.arrivals = a.hold == kHoldDecode ? 2 : 1;
  t.p = p;
  CUtensorMap k, v;
  if (!pages_map(&k, a.k_cache, a, kSlice) || !pages_map(&v, a.v_cache, a, kSlice)) return cudaErrorInvalidValue;
  Report rep = shape;
  rep.blocks[rep.set] = num_sms;
  const bool wide = G > 8;
#define DECODE_CASE(DD, F, W) \
  if (a.D == DD && (a.f16 != 0) == F && wide == W) return launch<DD, F, W>(t, k, v, rep, beside.prefix, num_sms, stream);
  DECODE_CASE(64, false, false)
  DECODE_CASE(64, false, true)
  DECODE_CASE(64, true, false)
  DECODE_CASE(64, true, true)
  DECODE_CASE(128, false, false)
  DECODE_CASE(128, false, true)
  DECODE_CASE(128, true, false)
  DECODE_CASE(128, true, true)
#undef DECODE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace attn
}  // namespace moe
