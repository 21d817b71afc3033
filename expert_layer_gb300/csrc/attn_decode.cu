// Attention of single tokens over the paged cache.
//
// A unit is one sequence's token on one key-value head: its G query heads
// (at most 16; larger groups make several units) share every key and value
// that is read.  The keys of all units form one line of 16-key slices (a
// slice lies within a page), cut into equal ranges for the blocks, so that
// lengths as different as 1 and 100,000 load the GPU evenly; a unit that
// spans blocks leaves one part per block and the merge kernel joins them.
//
// Bound: HBM (4 D bytes per key and key-value head against 4 G D flops).  In a
// block every warp works alone on slices w, w + 8, ... of the unit with its
// own softmax state, m, l and O in registers, and keeps its own ring of
// slices filled by TMA, across units: no barrier until the unit's end, where
// the eight states are joined.
//   S = Q K^T, O += P V   mma.sync m16n8k16, rows = heads (8 or 16 of 16)
#include "attn.h"
#include "attn_ptx.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kSlice = 16;          // keys
constexpr int kStages = 3;          // slices in flight per warp
constexpr float kLag = 8.0f;        // log2 of how far the maximum in use may lag

template <int D>
struct Shape {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalfBytes = kSlice * 128;                  // 2 KB: 16 keys x 64 elements
  static constexpr int kTileBytes = kHalves * kHalfBytes;          // K or V of a slice
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kRing = kStages * kStageBytes;              // of one warp
  static constexpr int kJoin = kWarps * kRing;                     // O of 8 rows, every warp
  static constexpr int kStats = kJoin + kWarps * 8 * D * 4;        // m and l of 16 rows, every warp
  static constexpr int kBars = kStats + kWarps * 16 * 2 * 4;
  static constexpr int kScan = kBars + kWarps * kStages * 8;
  static constexpr size_t kSmem = kScan + 256 + 1024;
};

// The units of one block: a cursor over (sequence, unit of the sequence),
// empty sequences left out.  `pos` is the unit's first slice on the line.
struct Cursor {
  int b, u, len, slices;
  long long pos;
};

struct DecodeArgs {
  AttnArgs a;
  float c;              // |scale| log2 e, > 0
  uint32_t flip;        // sign bits of two elements when the scale is negative
  int chunks;           // units per key-value head
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

// To the next unit that has slices (or past the last sequence).
__device__ __forceinline__ void advance(const DecodeArgs& t, Cursor& c, int units) {
  c.pos += c.slices;
  if (++c.u < units) return;
  c.u = 0;
  c.slices = 0;
  while (++c.b < t.a.n_seq) {
    c.len = seq_len(t.a, c.b);
    c.slices = slices_of(c.len);
    if (c.slices) break;
  }
}

template <int D, bool kF16, bool kWide>
__global__ void __launch_bounds__(kThreads, 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const DecodeArgs t, const Report rep) {
  using S = Shape<D>;
  constexpr int kRowSets = kWide ? 2 : 1;            // rows g and (wide) g + 8 of a thread
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* join = reinterpret_cast<float*>(smem + S::kJoin);
  float* stats = reinterpret_cast<float*>(smem + S::kStats);
  long long* scan = reinterpret_cast<long long*>(smem + S::kScan);     // [8] warp sums, then the start
  const AttnArgs& a = t.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.Hq / a.Hkv, units = a.Hkv * t.chunks;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars) + warp * kStages;
  unsigned char* ring = smem + warp * S::kRing;
  bool bad = false, late = false;

  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&bars[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }

  // --- the line of slices: every thread sums a run of sequences
  const int run = (a.n_seq + kThreads - 1) / kThreads;
  const int s0 = min(a.n_seq, (int)threadIdx.x * run), s1 = min(a.n_seq, s0 + run);
  long long mine = 0;
  for (int s = s0; s < s1; ++s) {
    const int n = a.kv_lens[s];
    if (blockIdx.x == 0 && (n < 0 || n > ((long long)a.table_pages << a.page_shift))) bad = true;
    mine += (long long)slices_of(seq_len(a, s)) * units;
  }
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  before += incl - mine;
  if (blockIdx.x == 0) {                     // the merge kernel reads where each sequence lies
    long long at = before;
    for (int s = s0; s < s1; ++s) {
      t.p.base[s] = at;
      at += (long long)slices_of(seq_len(a, s)) * units;
    }
    if (threadIdx.x == kThreads - 1) t.p.base[a.n_seq] = total;
  }
  const int blocks = decode_blocks(total, (long long)a.n_seq * units, gridDim.x);
  const long long start = total * blockIdx.x / blocks, end = total * (blockIdx.x + 1) / blocks;
  const bool work = (int)blockIdx.x < blocks && start < end;
  if (work && start >= before && start < before + mine) {
    long long at = before;
    for (int s = s0; s < s1; ++s) {
      const long long n = (long long)slices_of(seq_len(a, s)) * units;
      if (start < at + n) {
        scan[kWarps] = s;
        scan[kWarps + 1] = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();

  if (work) {
    Cursor cur;
    cur.b = (int)scan[kWarps];
    cur.len = seq_len(a, cur.b);
    cur.slices = slices_of(cur.len);
    cur.u = (int)((start - scan[kWarps + 1]) / cur.slices);
    cur.pos = scan[kWarps + 1] + (long long)cur.u * cur.slices;

    // --- loads: the same walk, a few slices ahead
    Cursor ld = cur;
    int ld_slice = (int)max(0ll, start - ld.pos) + warp;     // this warp's next slice of unit ld
    uint32_t issued = 0;
    int page = 0;
    // moves ld to this warp's next slice and fetches its page id; false: none left
    auto locate = [&]() {
      while (ld.pos < end) {
        if (ld_slice < min((long long)ld.slices, end - ld.pos)) {
          page = a.page_table[(long long)ld.b * a.table_pages + ((ld_slice * kSlice) >> a.page_shift)];
          return true;
        }
        advance(t, ld, units);
        ld_slice = warp;
      }
      return false;
    };
    bool more = locate();
    auto issue = [&]() {
      if (!more) return;
      if (lane == 0) {
        if ((unsigned)page >= (unsigned)a.pages) {
          bad = true;
          page = 0;
        }
        const int st = issued % kStages, row = (ld_slice * kSlice) & ((1 << a.page_shift) - 1);
        const int hk = ld.u / t.chunks;
        unsigned char* dst = ring + st * S::kStageBytes;
        mbar_expect_tx(&bars[st], S::kStageBytes);
#pragma unroll
        for (int hh = 0; hh < S::kHalves; ++hh)
          tma_load_4d(dst + hh * S::kHalfBytes, &tmK, hh * 64, row, hk, page, &bars[st]);
#pragma unroll
        for (int hh = 0; hh < S::kHalves; ++hh)
          tma_load_4d(dst + S::kTileBytes + hh * S::kHalfBytes, &tmV, hh * 64, row, hk, page, &bars[st]);
      }
      ++issued;
      ld_slice += kWarps;
      more = locate();
    };
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) issue();

    // ldmatrix source of this lane: K: 8x8 matrices (keys 0-7 | 8-15) x (d 0-7 | 8-15),
    // V transposed: the same with keys fastest; rows are swizzled by key % 8
    const int k_row = (lane & 7) + ((lane & 16) >> 1), k_col = (lane >> 3) & 1;
    const int v_row = (lane & 7) + (lane & 8), v_col = lane >> 4;
    const int quad = lane & 3, gq = lane >> 2;
    uint32_t used = 0;

    while (cur.pos < end) {
      const long long begin = max(0ll, start - cur.pos);
      const int first = (int)begin, last = (int)min((long long)cur.slices, end - cur.pos);
      const int hk = cur.u / t.chunks, h0 = hk * G + (cur.u - hk * t.chunks) * 16;
      const int rows = min(16, hk * G + G - h0);
      uint32_t q[D / 16][2 * kRowSets];
      {
        const uint16_t* src = a.q.data + (long long)cur.b * a.q.tok;
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
      }
      float o[D / 8][4];
      float m[kRowSets], l[kRowSets];
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
#pragma unroll
      for (int rs = 0; rs < kRowSets; ++rs) m[rs] = -INFINITY, l[rs] = 0.f;

      for (int s = first + warp; s < last; s += kWarps) {
        const int st = used % kStages;
        if (!late && !__all_sync(0xffffffffu, spin_wait(&bars[st], (used / kStages) & 1))) late = true;
        const uint32_t kb = smem_u32(ring + st * S::kStageBytes), vb = kb + S::kTileBytes;
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t r[4];
          const int chunk = (kk & 3) * 2 + k_col;
          ldsm4(kb + (kk >> 2) * S::kHalfBytes + k_row * 128 + ((chunk ^ (k_row & 7)) << 4), r);
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
          ldsm4_t(vb + (i >> 2) * S::kHalfBytes + v_row * 128 + ((chunk ^ (v_row & 7)) << 4), r);
          mma<kF16>(o[2 * i], p[0], p[1], p[2], p[3], r[0] & keep0, r[1] & keep1);
          mma<kF16>(o[2 * i + 1], p[0], p[1], p[2], p[3], r[2] & keep0, r[3] & keep1);
        }
        __syncwarp();            // every lane has read the stage
        ++used;
        issue();
      }

      // --- join the warps' states: row r is out = sum_w 2^{m_w - M} O_w / sum_w 2^{m_w - M} l_w
#pragma unroll
      for (int rs = 0; rs < kRowSets; ++rs) {
        l[rs] += __shfl_xor_sync(0xffffffffu, l[rs], 1);
        l[rs] += __shfl_xor_sync(0xffffffffu, l[rs], 2);
        if (quad == 0) {
          stats[(warp * 16 + gq + 8 * rs) * 2] = m[rs];
          stats[(warp * 16 + gq + 8 * rs) * 2 + 1] = l[rs];
        }
      }
      const bool whole = cur.pos >= start && cur.pos + cur.slices <= end;
      const int slot = 2 * blockIdx.x + (cur.pos < start ? 0 : 1);
#pragma unroll
      for (int rs = 0; rs < kRowSets; ++rs) {
        if (first + warp < last) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2*>(join + (warp * 8 + gq) * D + 8 * i + 2 * quad) =
                make_float2(o[i][2 * rs], o[i][2 * rs + 1]);
        }
        __syncthreads();
        const int live = min(kWarps, last - first);            // warps that had a slice
        for (int i = threadIdx.x; i < 8 * (D / 4); i += kThreads) {
          const int r8 = i / (D / 4), r = r8 + 8 * rs, d = (i % (D / 4)) * 4;
          if (r >= rows) continue;
          float M = -INFINITY;
          for (int w = 0; w < live; ++w) M = fmaxf(M, stats[(w * 16 + r) * 2]);
          float sum = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int w = 0; w < live; ++w) {
            const float f = M == -INFINITY ? 0.f : ex2(stats[(w * 16 + r) * 2] - M);
            sum = fmaf(f, stats[(w * 16 + r) * 2 + 1], sum);
            const float4 x = *reinterpret_cast<const float4*>(join + (w * 8 + r8) * D + d);
            v.x = fmaf(f, x.x, v.x);
            v.y = fmaf(f, x.y, v.y);
            v.z = fmaf(f, x.z, v.z);
            v.w = fmaf(f, x.w, v.w);
          }
          const float inv = 1.0f / sum;
          v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
          const float lse = M + lg2(sum);
          const long long row = (long long)cur.b * a.Hq + h0 + r;
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
        __syncthreads();
      }
      advance(t, cur, units);
    }
    // after a timeout: the loads already issued land before the block exits
    if (late && lane == 0)
      for (uint32_t i = issued > (uint32_t)kStages ? issued - kStages : 0; i < issued; ++i)
        mbar_wait(&bars[i % kStages], (i / kStages) & 1);
  }
  const int any_bad = __syncthreads_or(bad), any_late = __syncthreads_or(late);
  if (threadIdx.x == 0) report(rep, (any_bad ? kStatusBounds : 0) | (any_late ? kStatusTimeout : 0));
}

// ------------------------------------------------------------------ merge
// Rows whose keys were split: `splits` parts of the shared prefix (row order),
// and the row's own keys, which one block did whole (the row's part, or the
// final result when there is no prefix) or several (their slots, in the order
// of the blocks).  A warp per row.
template <int D, bool kF16>
__global__ void __launch_bounds__(128) decode_merge_kernel(const DecodeArgs t, int splits, int grid) {
  constexpr int N = D / 32;
  pdl_wait();   // programmatic dependent launch: the parts are complete
  const AttnArgs& a = t.a;
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)a.T * a.Hq;
  const long long row = (long long)blockIdx.x * 4 + threadIdx.x / 32;
  if (row >= rows) return;
  const int b = (int)(row / a.Hq), h = (int)(row % a.Hq), G = a.Hq / a.Hkv;
  const int units = a.Hkv * t.chunks, u = (h / G) * t.chunks + (h % G) / 16, r = (h % G) % 16;
  const long long total = t.p.base[a.n_seq], b0 = t.p.base[b], n = (t.p.base[b + 1] - b0) / units;
  int c0 = 0, own = 0;                       // blocks c0 .. c0 + own - 1 hold the row's own keys
  long long start0 = 0;
  const long long ub = b0 + u * n;
  if (n > 0) {
    const long long blocks = decode_blocks(total, (long long)a.n_seq * units, grid);
    c0 = (int)(((ub + 1) * blocks - 1) / total);
    own = (int)(((ub + n) * blocks - 1) / total) - c0 + 1;
    start0 = total * c0 / blocks;
  }
  if (splits == 0 && own == 1) return;       // final already
  // part i < splits: the prefix; then the own parts
  auto where = [&](int i, const float*& o, const float*& lse) {
    if (i < splits || own == 1) {
      const long long at = (long long)i * rows + row;   // the row's own part follows the prefix's
      o = t.p.tc_o + at * D;
      lse = t.p.tc_lse + at;
    } else {
      const int c = c0 + i - splits;
      const long long at = (2ll * c + (c == c0 && ub >= start0 ? 1 : 0)) * 16 + r;
      o = t.p.slot_o + at * D;
      lse = t.p.slot_lse + at;
    }
  };
  const int parts = splits + own;
  float top = -INFINITY;
  for (int i = lane; i < parts; i += 32) {
    const float *o, *lse;
    where(i, o, lse);
    top = fmaxf(top, *lse);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  float acc[N], sum = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.f;
  if (top != -INFINITY) {
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      const float *o, *lse;
      where(i, o, lse);
      const float w = ex2(*lse - top);
      sum += w;
      if (w != 0.f) {
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = fmaf(w, o[lane * N + j], acc[j]);
      }
    }
  }
  const float inv = sum > 0.f ? 1.0f / sum : sum;       // no keys: 0; NaN stays
#pragma unroll
  for (int j = 0; j < N; ++j) a.out[row * D + lane * N + j] = kF16 ? f2h(acc[j] * inv) : f2bf(acc[j] * inv);
  if (a.lse && lane == 0) a.lse[row] = sum == 0.f ? -INFINITY : (top + lg2(sum)) * 0.693147180559945f;
}

template <int D, bool kF16, bool kWide>
cudaError_t launch(const DecodeArgs& t, const CUtensorMap& k, const CUtensorMap& v, const Report& rep, int splits,
                   int grid, cudaStream_t stream) {
  auto kern = attn_decode_kernel<D, kF16, kWide>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<D>::kSmem);
  if (err != cudaSuccess) return err;
  kern<<<grid, kThreads, Shape<D>::kSmem, stream>>>(k, v, t, rep);
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const long long rows = (long long)t.a.T * t.a.Hq;
  return launch_pdl(decode_merge_kernel<D, kF16>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, stream, t, splits,
                    grid);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnArgs& a, int splits, const DecodeParts& p, const Report& shape, int num_sms,
                               cudaStream_t stream) {
  DecodeArgs t{};
  t.a = a;
  t.c = (a.scale < 0 ? -a.scale : a.scale) * 1.4426950408889634f;
  if (t.c < 1.2e-38f) t.c = 1.2e-38f;      // a masked logit of -inf stays one
  t.flip = a.scale < 0 ? 0x80008000u : 0u;
  const int G = a.Hq / a.Hkv;
  t.chunks = (G + 15) / 16;
  t.p = p;
  CUtensorMap k, v;
  if (!kv_map(&k, a, a.k_cache, a.k, kSlice) || !kv_map(&v, a, a.v_cache, a.v, kSlice)) return cudaErrorInvalidValue;
  Report rep = shape;
  rep.blocks[rep.set] = num_sms;
  const bool wide = G > 8;
#define DECODE_CASE(DD, F, W) \
  if (a.D == DD && (a.f16 != 0) == F && wide == W) return launch<DD, F, W>(t, k, v, rep, splits, num_sms, stream);
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
