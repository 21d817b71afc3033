// Attention of many rows on the tensor cores: whole prompts, chunks of them
// over the paged cache, and the shared prefix of a decode batch.
//
// A tile is 128 rows of one key-value head: `tt` tokens x G query heads
// (tt = 128 / G, row = token * G + head), so that the G heads of a group
// share every key and value tile.  A block takes two tiles (2 tt tokens of one
// sequence) through the visible keys in blocks of 128:
//   S = Q K^T                      tcgen05.mma, fp32 in tensor memory
//   m' = max(m, max_j c S_j)       c = scale log2(e)
//   P = 2^{c S - m'},  l += sum P  fp32; P rounded to the element type for
//   O += P V                       the second product (A from tensor memory)
// with out = O / l and lse = (m + log2 l) ln 2 at the end.  m is a scale, not
// the exact maximum: a row takes the maximum of its first few logits, and P is
// formed with it from then on, without looking at the logits first.  The sum of
// P, needed anyway, says when a row has outgrown its scale (2^15: P stays within
// f16, and bf16 rounds relative to P whatever its size); only then the row's
// maximum is taken again and l and O are rescaled, which hardly happens.  A row
// whose logits are all -inf so far has no scale (m = -inf) and takes the path
// that looks at every logit.
//
// Rounding P to the element type is the price of the second product on the
// tensor cores: the outputs' error against 64 bits (relative, over all outputs)
// is 2.3e-3 where weights in 32 bits leave 1.7e-3, the rounding of the output
// (bf16; f16 2.9e-4 and 2.1e-4).  l sums P before that, for the log-sums and the
// joins of parts; dividing by a second sum, of the rounded P, so that the
// rounding of a dominant key cancels, gave 2.1e-3 (2.5e-4) and took 3 to 11%
// more time (8192 causal 313 -> 344 us, 16 prompts of 512 tokens 50.8 -> 56.4).
//
// Bound: D = 128, the tensor pipe (512 cycles for each of a tile's two products
// per key block, 2048 for both tiles, of a period of ~2550); D = 64, the chain
// product - softmax - product of two tiles in turns (~2400, the products half as
// long).  Two tiles make one of them run while the other waits for its barriers,
// and fill tensor memory.  Exponentials (32 a cycle and SM: 1024 per period) are
// not the bound: a quarter of them as a polynomial on the FMA pipe took 375 us
// for 8192 tokens where the kernel of that time took 324.
// Measured (32 query and 4 key-value heads of 128, bf16): 8192 tokens causal
// 313 us in bursts of a few calls = 1.75 PFLOP/s, 91% of the library's matrix
// product (345 after seconds, under the power cap, 93% of its rate then); 8192 x
// 8192 598 us = 1.84; 16 prompts of 512 tokens 51 us, 64 of 128 35.5 (an item of
// one block is a chain of ~4.2 us: product 0.2, softmax 1.3, product 0.7,
// epilogue 1.6).
#include <cuda.h>

#include "attn.h"
#include "attn_ptx.cuh"

namespace moe {
namespace attn {
namespace {

using namespace tcx;

constexpr int kRows = 128;          // rows of a tile
constexpr int kKeys = 128;          // keys of a block
constexpr int kItems = 4;           // ring of work items
constexpr int kAskAhead = 3;        // key blocks before an item's end at which the next one is asked for
constexpr int kSoftWarps = 8;       // two tiles x four warps, one row per thread
constexpr int kThreads = (kSoftWarps + 4) * 32;
// Registers per thread: 168 at launch (three warpgroups); the softmax
// warpgroups, which hold a row of 128 logits, draw on the third one's.
constexpr int kSoftRegs = 208, kLoadRegs = 88;
static_assert(2 * kSoftRegs + kLoadRegs <= 3 * 168, "the shares come from the launch's registers");
constexpr int kHalf = kKeys / 2;
constexpr float kMost = 32768.0f;   // sum of a row's P over half a block that asks for a new scale
constexpr uint32_t kTmemCols = 512;

// Tiles in shared memory: rows of 64 elements in 1 KB swizzle atoms of 8.  Q,
// and K and V from packed rows: one column of atoms after the other.  K and V
// from pages: atoms of the same 8 rows side by side (pages_map).
template <int D, bool kPaged>
struct Shape {
  static constexpr int kHalves = D / 64;                       // 128-byte wide swizzled columns
  static constexpr int kHalfBytes = kRows * 128;               // 16 KB: a column
  static constexpr int kColumn = kPaged ? 1024 : kHalfBytes;   // from a K or V column to the next
  static constexpr int kGroup = kPaged ? kHalves * 1024 : 1024;   // from 8 rows of K or V to the next
  static constexpr int kTileBytes = kHalves * kHalfBytes;      // a Q, K or V tile
  // ring of K and V tiles: 8192 causal with 3 and 4 stages of 32 KB 421 and 324 us
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kRing = 2 * kTileBytes;                 // the ring follows the two Q tiles
  static constexpr int kOut = kRing + kStages * kTileBytes;    // 32 rows of 128 bytes per softmax warp
  static constexpr int kBars = kOut + kSoftWarps * 32 * 128;
  static constexpr size_t kSmem = kBars + 1024;
};

struct Item {
  int row0;        // first token row of tile 0; -1: no more items
  int tok[2];      // tokens of the two tiles
  int n[2];        // key blocks of the two tiles
  int head;        // key-value head
  int b0;          // first key block
  int len;         // keys of the sequence
  int seen;        // keys that token row0 sees (causal; may be <= 0), else len
  int split;
};

// Arrivals that the barriers wait for, one too many where a test holds one
struct Arrivals {
  int keys, stage, query, s, p, o, half, turn, item, next;
  Arrivals(int hold = kHoldNone)
      : keys(1 + (hold == kHoldKeys)), stage(2 + (hold == kHoldStage)), query(1 + (hold == kHoldQuery)),
        s(1 + (hold == kHoldS)), p(4 + (hold == kHoldP)), o(1 + (hold == kHoldO)), half(1 + (hold == kHoldHalf)),
        turn(4 + (hold == kHoldTurn)), item(1 + (hold == kHoldItem)), next(1 + (hold == kHoldNext)) {}
};

struct TcAttnArgs {
  AttnArgs a;
  int G;                         // Hq / Hkv
  Divisor by_splits, by_Hkv, by_per, by_G;
  int tt, slots, splits;
  int box;                       // rows of a K / V box
  float c;                       // scale log2 e, not 0
  float hidden;                  // a masked logit: c times it is -inf
  int out_box;                   // 32 rows of a tile are whole heads of whole tokens
  float* part_o;                 // [splits, T, Hq, D], null when the result is final
  float* part_lse;               // [splits, T, Hq], log2
  Arrivals arrivals;
};

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
      "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Keys [keys][D] as the B operand of S = Q K^T: K-major, 128-byte swizzle,
// groups of 8 keys `group` bytes apart.
__device__ __forceinline__ uint64_t umma_desc_k(uint32_t saddr, uint32_t group) {
  return (umma_desc(saddr) & ~((uint64_t)0x3FFF << 32)) | (uint64_t)(group >> 4) << 32;
}
// Values [keys][D] as the B operand of O += P V: D-major ("transposed"),
// 128-byte swizzle; the next 64 columns of D `column` bytes on (leading
// offset), the next 8 keys `group` bytes on (stride offset).
__device__ __forceinline__ uint64_t umma_desc_v(uint32_t saddr, uint32_t column, uint32_t group) {
  return (umma_desc_k(saddr, group) & ~((uint64_t)0x3FFF << 16)) | (uint64_t)(column >> 4) << 16;
}
__device__ __forceinline__ void umma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accum));
}
// kind::f16 with fp32 accumulators; b_t: B is N-major
template <bool kF16>
__device__ __forceinline__ constexpr uint32_t idesc_of(int n, bool b_t) {
  return (1u << 4) | ((kF16 ? 0u : 1u) << 7) | ((kF16 ? 0u : 1u) << 10) | ((b_t ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}

// ------------------------------------------------------------------ work items
// Sequence s owns the tile slots base(s) .. base(s+1) - 1 with base(s) =
// floor(q_starts[s] / (2 tt)) + s: at least as many as it has tiles, without a
// prefix sum over the batch.  All lanes of the warp search together.
__device__ __forceinline__ int find_seq(const AttnArgs& a, const Divisor& per, int slot) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.n_seq;                       // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int s = lo + lane * step;
    const bool at = lane * step < n && per.of(max(0, a.q_starts[s])) + s <= slot;
    const int hit = 31 - __clz((int)(__ballot_sync(0xffffffffu, at) | 1u));
    lo += hit * step;
    n = min(step, n - hit * step);
  }
  return lo;
}

// Item `idx` (warp-uniform); false when its slot has no rows.  Later tiles of
// a sequence see more keys: they come first.
__device__ __forceinline__ bool make_item(const TcAttnArgs& t, int idx, Item& it, int& seq, int& k0) {
  const AttnArgs& a = t.a;
  const int unit = t.by_splits.of(idx), back = t.by_Hkv.of(unit);
  it.split = idx - unit * t.splits;
  it.head = unit - back * a.Hkv;
  const int slot = t.slots - 1 - back;
  const int per = 2 * t.tt;
  int q0 = 0, q1 = a.T, tile = slot;
  seq = 0;
  if (a.q_starts) {
    seq = find_seq(a, t.by_per, slot);
    q0 = a.q_starts[seq];
    q1 = a.q_starts[seq + 1];
    tile = slot - (t.by_per.of(max(0, q0)) + seq);
    if (q0 < 0 || q1 < q0 || q1 > a.T || tile < 0) return false;
  }
  const long long first = (long long)tile * per;
  if (first >= q1 - q0) return false;
  it.row0 = q0 + (int)first;
  const int left = q1 - it.row0;
  it.tok[0] = min(left, t.tt);
  it.tok[1] = max(0, min(left - t.tt, t.tt));
  k0 = 0;
  if (a.prefix_table) {
    it.len = a.prefix_len;
  } else if (a.page_table) {
    it.len = a.kv_lens[seq];
    if (it.len < 0 || it.len > ((long long)a.table_pages << a.page_shift)) it.len = 0;
  } else {
    k0 = a.kv_starts[seq];
    it.len = a.kv_starts[seq + 1] - k0;
    if (k0 < 0 || it.len < 0 || k0 > a.Tk - it.len) k0 = 0, it.len = 0;
  }
  it.seen = a.causal ? it.len - (q1 - q0) + (int)first + 1 : it.len;
  int nb[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    int v = a.causal ? it.seen + x * t.tt + it.tok[x] - 1 : it.len;   // keys the tile's last token sees
    v = min(v, it.len);
    nb[x] = it.tok[x] > 0 && v > 0 ? (v + kKeys - 1) / kKeys : 0;
  }
  const int all = max(nb[0], nb[1]);
  // floor(all * split / splits), and the same of split + 1
  const int whole = t.by_splits.of(all), more = all - whole * t.splits;
  it.b0 = whole * it.split + t.by_splits.of(more * it.split);
  const int b1 = whole * (it.split + 1) + t.by_splits.of(more * (it.split + 1));
#pragma unroll
  for (int x = 0; x < 2; ++x) it.n[x] = max(0, min(nb[x], b1) - it.b0);
  return true;
}

// Index arrays of the call, checked once (by the warp that has item 0): what is
// out of order is reported here and skipped or clamped where it is used.
__device__ __forceinline__ bool bad_arrays(const AttnArgs& a) {
  bool bad = a.q_starts && (a.q_starts[0] != 0 || a.q_starts[a.n_seq] != a.T);      // rows of no sequence
  if (a.q_starts)
    for (int s = threadIdx.x & 31; s < a.n_seq; s += 32) {
      const int q0 = a.q_starts[s], q1 = a.q_starts[s + 1];
      bad |= q0 < 0 || q1 < q0 || q1 > a.T;
      if (!a.page_table) {
        const int k0 = a.kv_starts[s], k1 = a.kv_starts[s + 1];
        bad |= k0 < 0 || k1 < k0 || k1 > a.Tk;
      } else {
        const int n = a.kv_lens[s];
        bad |= n < 0 || n > ((long long)a.table_pages << a.page_shift);
      }
    }
  return bad;
}

// ------------------------------------------------------------------ the kernel
// warps 0-3, 4-7   softmax and epilogue of tile 0 and 1 (thread = row)
// warp 8           work items, TMA loads of Q, K and V
// warps 9, 10      issue the MMAs of tile 0 and 1 (warp 11 only completes the
//                  warpgroup): per key block O += P V, half by half as P
//                  comes, then S = Q K' of the next block; one tile's softmax
//                  runs while the other multiplies.  A barrier costs an
//                  issuing warp ~200 cycles even when it is complete (the MMAs'
//                  operands fill the shared-memory pipe), which one warp for
//                  both tiles spent with the tensor core idle.
// Tensor memory: S0 | S1 | O0 | O1; P overwrites the first half of its S.
// One thread issues all MMAs of a tile, in order: a commit after S(j+1) also
// covers O += P(j) V, so a softmax warp that has S(j+1) may rescale O without
// waiting.
template <int D, bool kF16, bool kPaged>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, const TcAttnArgs t,
                   const Report rep) {
  using S = Shape<D, kPaged>;
  constexpr int NS = S::kStages;
  extern __shared__ __align__(1024) unsigned char smem[];      // swizzle atoms of 1 KB
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t* kv_empty = kv_full + NS;
  uint64_t* q_full = kv_empty + NS;
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_empty + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 4;         // p_full: [tile][half]
  uint64_t* h_done = o_full + 2;         // [tile]: the product with the first half of a block
  uint64_t* turn = h_done + 2;           // [tile]: its softmax may begin a block
  uint64_t* it_full = turn + 2;
  uint64_t* it_empty = it_full + kItems;
  uint64_t* drain = it_empty + kItems;
  uint64_t* clc = drain + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(clc + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  Item* ring = reinterpret_cast<Item*>(clc + 2);
  uint4* answer = reinterpret_cast<uint4*>(smem + S::kBars + 1024 - 16);

  const AttnArgs& a = t.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = t.G;
  if (threadIdx.x == 0) {
    prefetch_map(&tmQ);
    prefetch_map(&tmK);
    prefetch_map(&tmV);
    prefetch_map(&tmO);
  }
  pdl_trigger();   // a merge kernel, or the decode kernel beside it, may become resident

  if (threadIdx.x == 0) {
    const Arrivals& n = t.arrivals;
    for (int s = 0; s < NS; ++s) { mbar_init(&kv_full[s], s ? 1 : n.keys); mbar_init(&kv_empty[s], n.stage); }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], n.query);
      mbar_init(&q_empty[x], 1);
      mbar_init(&s_full[x], n.s);
      mbar_init(&p_full[2 * x], n.p);
      mbar_init(&p_full[2 * x + 1], n.p);
      mbar_init(&o_full[x], n.o);
      mbar_init(&h_done[x], n.half);
      mbar_init(&turn[x], n.turn);
    }
    for (int i = 0; i < kItems; ++i) { mbar_init(&it_full[i], n.item); mbar_init(&it_empty[i], kSoftWarps + 2); }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    mbar_init(clc, n.next);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == kSoftWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  bool bad = false;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    if (warp == kSoftWarps) {
    // ------------------------------------------------------------ producer
    uint32_t kv = 0, nq[2] = {0, 0}, ni = 0;    // loads issued, items published
    bool ok = true;
    const int boxes = kKeys / t.box;            // boxes of a full K or V tile (per 64 columns)
    // The grid has a block per item; a running block takes over blocks that have
    // not started (cluster launch control), so the items balance themselves.
    // It asks for the next one while the last loads of an item are issued.
    int idx = blockIdx.x;
    uint32_t asked = 0;
    auto ask = [&]() {
      if (lane == 0) {
        mbar_expect_tx(clc, 16);
        asm volatile(
            "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                smem_u32(answer)),
            "r"(smem_u32(clc))
            : "memory");
      }
      ++asked;
    };
    auto answered = [&]() {                       // the block asked for, -1: none is left
      int next = -1;
      asm volatile(
          "{\n .reg .b128 r;\n .reg .pred p;\n .reg .b32 y, z, w;\n ld.shared.b128 r, [%1];\n"
          " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
          " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, r;\n}\n"
          : "+r"(next)
          : "r"(smem_u32(answer))
          : "memory");
      return next;
    };
    auto taken = [&]() {
      ok = warp_spin(clc, (asked - 1) & 1);
      const int next = answered();
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      return ok ? next : -1;
    };
    while (ok) {
      const bool end = idx < 0;
      Item it;
      int seq = 0, k0 = 0;
      if (!end) {
        if (idx != (int)blockIdx.x && lane == 0) report(rep, idx, 0);
        if (idx == 0) bad |= bad_arrays(a);
        if (!make_item(t, idx, it, seq, k0)) {
          ask();
          idx = taken();
          continue;
        }
      } else {
        it = Item{};
        it.row0 = -1;
      }
      const int32_t* list = nullptr;
      if (kPaged) list = a.prefix_table ? a.prefix_table : a.page_table + (long long)seq * a.table_pages;
      // page of this lane's box in block b (lanes 0 .. boxes-1)
      auto fetch = [&](int b) {
        const int key = b * kKeys + lane * t.box;
        return kPaged && lane < boxes && key < it.len ? list[key >> a.page_shift] : 0;
      };
      auto checked = [&](int p) {
        if (!kPaged || (unsigned)p < (unsigned)a.pages) return p;
        bad = true;
        return 0;
      };
      int page = it.n[0] + it.n[1] > 0 && !end ? fetch(it.b0) : 0;       // under way while Q is loaded
      const int slot = ni % kItems;
      if (!warp_spin(&it_empty[slot], ((ni / kItems) & 1) ^ 1)) { ok = false; break; }
      if (lane == 0) {
        ring[slot] = it;
        mbar_arrive(&it_full[slot]);
      }
      ++ni;
      if (end) break;
      const int n = max(it.n[0], it.n[1]);
      if (n <= kAskAhead) ask();
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (ok && it.n[x] > 0) {
          ok = warp_spin(&q_empty[x], (nq[x] & 1) ^ 1);
          if (ok && lane == 0) {
            mbar_expect_tx(&q_full[x], (uint32_t)(S::kHalves * G * t.tt * 128));
            for (int hh = 0; hh < S::kHalves; ++hh)
              tma_load_3d(smem + x * S::kTileBytes + hh * S::kHalfBytes, &tmQ, hh * 64, it.head * G,
                          it.row0 + x * t.tt, &q_full[x]);
          }
          if (ok) ++nq[x];
        }
      for (int j = 0; j < n && ok; ++j) {
        const int b = it.b0 + j;
        page = checked(page);
        const int next = j + 1 < n ? fetch(b + 1) : 0;
        if (j > 0 && n - j == kAskAhead) ask();
        // boxes that hold keys of the sequence; the rest of the tile is not read
        const int nbox = min(boxes, (it.len - b * kKeys + t.box - 1) / t.box);
#pragma unroll 1
        for (int w = 0; w < 2; ++w, ++kv) {
          const int s = kv % NS;
          ok = warp_spin(&kv_empty[s], ((kv / NS) & 1) ^ 1);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(&kv_full[s], (uint32_t)(S::kHalves * nbox * t.box * 128));
          __syncwarp();
          if (lane < nbox) {
            unsigned char* dst = smem + S::kRing + s * S::kTileBytes;
            const int key = b * kKeys + lane * t.box;
            if (kPaged) {
              tma_load_5d(dst + lane * (t.box / 8) * S::kGroup, w ? &tmV : &tmK, 0, 0, 0,
                          (key & ((1 << a.page_shift) - 1)) / 8, page * a.Hkv + it.head, &kv_full[s]);
            } else {
#pragma unroll
              for (int hh = 0; hh < S::kHalves; ++hh)
                tma_load_3d(dst + hh * S::kHalfBytes, w ? &tmV : &tmK, hh * 64, k0 + key, it.head, &kv_full[s]);
            }
          }
        }
        page = next;
      }
      if (*(volatile int*)abort_flag) ok = false;
      if (ok) idx = taken();
    }
    if (lane == 0) {
      if (!ok) {
        atomicOr(abort_flag, 1);
        // the block asked for last is run by nobody: its word is written here
        if (asked && spin_wait(clc, (asked - 1) & 1)) {
          const int next = answered();
          if (next >= 0) report(rep, next, kStatusTimeout);
        }
      }
      // The loads issued land before the block exits, also where another warp
      // gives up after this one's last item (in normal use they are all used).
      for (uint32_t i = kv > (uint32_t)NS ? kv - NS : 0; i < kv; ++i) spin_wait(&kv_full[i % NS], (i / NS) & 1);
      for (int x = 0; x < 2; ++x)
        if (nq[x]) spin_wait(&q_full[x], (nq[x] - 1) & 1);
    }
    __syncwarp();
    } else if (warp <= kSoftWarps + 2) {
    // ------------------------------------------------------------ MMA issuers
    // The whole warp runs the loop on values that are uniform to the compiler
    // (constants, loop counters, results of warp reductions); one elected lane
    // issues.
    constexpr uint32_t kIdS = idesc_of<kF16>(kKeys, false), kIdO = idesc_of<kF16>(D, true);
    const int x = __reduce_max_sync(0xffffffffu, warp - kSoftWarps - 1);      // tile
    const uint32_t tS = x * kKeys, tO = 2 * kKeys + x * D;   // all 512 columns: the allocation starts at 0
    const uint32_t sQ = smem_u32(smem) + x * S::kTileBytes, sR = smem_u32(smem) + S::kRing;
    int ks = 0;                      // ring stage and phase of the next K tile; V tiles alternate with K tiles
    uint32_t kph = 0, ni = 0, qph = 0, pph = 0;
    bool ok = true;
    auto product_s = [&](int s) {
      if (elect_one()) {
        const uint64_t dq = umma_desc(sQ), dk = umma_desc_k(sR + s * S::kTileBytes, S::kGroup);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_bf16_id(tS, dq + (((kk / 4) * S::kHalfBytes + (kk % 4) * 32) >> 4),
                       dk + (((kk / 4) * S::kColumn + (kk % 4) * 32) >> 4), kIdS, kk ? 1u : 0u);
        umma_commit(&s_full[x]);
      }
      __syncwarp();
    };
    // one half (64 keys) of a block
    auto product_o = [&](int half, int s, uint32_t add) {
      if (elect_one()) {
        const uint64_t dv = umma_desc_v(sR + s * S::kTileBytes, S::kColumn, S::kGroup);
#pragma unroll
        for (int i = 0; i < kKeys / 32; ++i) {
          const int kk = half * (kKeys / 32) + i;
          umma_ts(tO, tS + kk * 8, dv + ((kk * 2 * S::kGroup) >> 4), kIdO, kk ? 1u : add);
        }
        if (half == 0) umma_commit(&h_done[x]);
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) umma_commit(bar);
      __syncwarp();
    };
    auto next = [&](int s, uint32_t ph, int by, int& s2, uint32_t& ph2) {
      s2 = s + by;
      ph2 = ph;
      if (s2 >= NS) s2 -= NS, ph2 ^= 1;
    };
    while (ok) {
      const int slot = ni % kItems;
      ok = warp_spin(&it_full[slot], (ni / kItems) & 1);
      if (!ok) break;
      const int row0 = __reduce_max_sync(0xffffffffu, ring[slot].row0);
      const int n0 = __reduce_max_sync(0xffffffffu, ring[slot].n[0]);
      const int n1 = __reduce_max_sync(0xffffffffu, ring[slot].n[1]);
      if (lane == 0) mbar_arrive(&it_empty[slot]);
      __syncwarp();
      ++ni;
      if (row0 < 0) break;
      const int n = max(n0, n1), nx = x ? n1 : n0;
      if (n == 0) continue;
      ok = warp_spin(&kv_full[ks], kph);
      if (ok && nx > 0) {
        ok = warp_spin(&q_full[x], qph);
        qph ^= 1;
        tc_fence_after();
        if (ok) product_s(ks);
        if (ok && nx == 1) commit(&q_empty[x]);
      }
      if (!ok) break;
      commit(&kv_empty[ks]);
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        int vs, k2;                  // V of this block, K of the next
        uint32_t vph, k2ph;
        next(ks, kph, 1, vs, vph);
        next(ks, kph, 2, k2, k2ph);
        // also for blocks that only the other tile has: a stage is given back
        // for the phase that it is in
        ok = warp_spin(&kv_full[vs], vph) && (j + 1 >= n || warp_spin(&kv_full[k2], k2ph));
        if (ok && j < nx) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!ok) continue;
            ok = warp_spin(&p_full[2 * x + half], pph);
            tc_fence_after();
            if (ok) product_o(half, vs, j > 0 ? 1u : 0u);
          }
          pph ^= 1;
          if (ok && j + 1 < nx) {
            product_s(k2);
            if (j + 2 == nx) commit(&q_empty[x]);
          } else if (ok) {
            commit(&o_full[x]);
          }
        }
        if (!ok) break;
        commit(&kv_empty[vs]);
        if (j + 1 < n) commit(&kv_empty[k2]);
        ks = k2;
        kph = k2ph;
      }
      if (*(volatile int*)abort_flag) ok = false;
    }
    // the MMAs issued finish before their memory is freed, whoever gives up
    if (!ok && lane == 0) atomicOr(abort_flag, 1);
    commit(&drain[x]);
    if (lane == 0) spin_wait(&drain[x], 0);
    __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ------------------------------------------------------------ softmax, epilogue
    const int x = warp >> 2;                                   // tile
    const int row = (warp & 3) * 32 + lane;                    // row of the tile
    const int token = t.by_G.of(row), g = row - token * G;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + x * kKeys, tO = tmem + lanes + 2 * kKeys + x * D;
    uint32_t ni = 0, ns = 0, no = 0, nt = 0, kv = 0;
    bool ok = true;
    while (ok) {
      const int slot = ni % kItems;
      if (!warp_spin(&it_full[slot], (ni / kItems) & 1)) { ok = false; break; }
      const Item it = ring[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&it_empty[slot]);
      ++ni;
      if (it.row0 < 0) break;
      const int n = x ? it.n[1] : it.n[0];
      // blocks that the tiles take in turns, and after which half
      const int shared = min(it.n[0], it.n[1]), both = shared > 1 ? shared : 0;
      const int turn_half = D == 64 || shared <= 16 ? 0 : 1;
      const uint32_t kv0 = kv;
      kv += 2 * max(it.n[0], it.n[1]);
      // keys that this row sees
      const int vis = a.causal ? min(it.seen + x * t.tt + token, it.len) : it.len;
      const bool live = token < (x ? it.tok[1] : it.tok[0]);
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++ns) {
        if (!warp_spin(&s_full[x], ns & 1)) { ok = false; break; }
        tc_fence_after();
        // Turns: left alone the two tiles fall into step, with the tensor core
        // idle while both compute P and the reverse (8192 x 8192 keys, D = 128:
        // 668 us).  A tile hands over when all its P is formed (594 us; after
        // the first half 622) or, where its MMAs are shorter (D = 64) or its
        // blocks few (16 prompts of 512 tokens 55.0 us instead of 60.3), after
        // the first half.
        if (j < both && !warp_spin(&turn[x], (nt & 1) ^ (x ? 0 : 1))) { ok = false; break; }
        const int b = it.b0 + j;
        const uint64_t c2 = pair(t.c, t.c);
        auto arrive = [&](int half) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * x + half]);
        };
        auto hand_over = [&](int half) {
          if (half == turn_half && j < both) {
            ++nt;
            if (lane == 0) mbar_arrive(&turn[x ^ 1]);
          }
        };
        const int lim = vis - b * kKeys;    // keys of the block that the row sees: more in later rows
        const int lim0 = __shfl_sync(0xffffffffu, lim, 0), lim1 = __shfl_sync(0xffffffffu, lim, 31);
        bool unset = __any_sync(0xffffffffu, live && m == -INFINITY && lim > 0);
        if (unset) {
          // a first scale: the maximum of the first few logits (all of them
          // -inf, as a product past fp32 or an infinity in a key makes them: the
          // loop below, which looks at every logit)
          float u[16];
          tmem_ld16(tS, *reinterpret_cast<uint32_t(*)[16]>(u));
          tmem_wait_ld();
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < 16; ++k) top = fmaxf(top, k < lim ? u[k] * t.c : -INFINITY);
          if (m == -INFINITY) m = top;
          unset = __any_sync(0xffffffffu, live && m == -INFINITY);
        }
        // 64 logits to P with the scale in use; the sum
        auto form = [&](const float (&s)[kHalf], uint32_t (&p)[32]) {
          const float off = m == -INFINITY ? 0.f : -m;
          const uint64_t off2 = pair(off, off);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const uint64_t y = fma2(pair(s[2 * k], s[2 * k + 1]), c2, off2);
            const float p0 = ex2(lo(y)), p1 = ex2(hi(y));
            sum[k & 1] = add2(sum[k & 1], pair(p0, p1));
            p[k] = pack2<kF16>(p0, p1);
          }
          sum[0] = add2(sum[0], sum[1]);
          return lo(sum[0]) + hi(sum[0]);
        };
        // A block that the warp's rows see whole: both halves written out,
        // without a look at the logits first and without branches (those of a
        // mask cost 10% over 8192 keys).
        int slow = 0;                       // first half that is left to the loop below
        if (lim0 >= kKeys && !unset) {
          float s0[kHalf], s1[kHalf];
          uint32_t p[32];
          tmem_ld64(tS, s0);
          tmem_wait_ld64(s0);
          tmem_ld64(tS + kHalf, s1);        // on its way meanwhile
          float sum = form(s0, p);
          tmem_wait_ld64(s1);
          if (!__any_sync(0xffffffffu, live && sum > kMost)) {
            l += sum;
            tmem_st32(tS, p);
            arrive(0);
            hand_over(0);
            sum = form(s1, p);
            slow = 1;
            if (!__any_sync(0xffffffffu, live && sum > kMost)) {
              hand_over(1);
              l += sum;
              tmem_st32(tS + 32, p);
              arrive(1);
              slow = 2;
            }
          }
        }
        // Blocks with masked keys, and rows that outgrew their scale or have none: a loop
        // over the halves, one piece of code.  (Code that does not stay in the
        // instruction cache costs ~100 cycles per eight instructions: with the
        // rare cases written out twice a first block took 3500 cycles.)
        // Rows of V past the keys' end hold other data (or NaN), which a weight
        // of 0 does not silence: clear them (each tile that multiplies them).
        const int tail = it.len - b * kKeys;
        if (tail < kKeys) {
          const uint32_t i = kv0 + 2 * j + 1;
          if (!warp_spin(&kv_full[i % NS], (i / NS) & 1)) { ok = false; break; }
          if (row >= tail) {
            uint4* v = reinterpret_cast<uint4*>(smem + S::kRing + (i % NS) * S::kTileBytes + (row / 8) * S::kGroup +
                                                (row % 8) * 128);
#pragma unroll 4
            for (int u = 0; u < S::kHalves * 8; ++u) v[(u / 8) * (S::kColumn / 16) + u % 8] = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
#pragma unroll 1
        for (int half = slow; half < 2; ++half) {
          const int from = half * kHalf;
          uint32_t p[32];
          if (lim1 <= from) {                                        // no row sees a key of it
#pragma unroll
            for (int k = 0; k < 32; ++k) p[k] = 0;
          } else {
            float s[kHalf];
            tmem_ld64(tS + from, s);
            tmem_wait_ld64(s);
#pragma unroll
            for (int k = 0; k < kHalf; ++k) s[k] = from + k < lim ? s[k] : t.hidden;
            float sum;
#pragma unroll 1
            for (int pass = 0;; ++pass) {
              sum = form(s, p);
              const bool need = live && (sum > kMost || (m == -INFINITY && lim > from));
              if (pass || !__any_sync(0xffffffffu, need)) break;
              // a new scale for the rows that need one: their maximum
              float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int k = 0; k < kHalf; ++k) mx[k & 3] = fmaxf(mx[k & 3], s[k] * t.c);
              const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
              const bool up = need && top > m;
              const float f = up ? ex2(m - top) : 1.0f;              // m = -inf: 0
              if (up) m = top;
              l *= f;
              if (j + half > 0) {
                // O += P V of the block before is complete (S of this one came
                // after it), that of the first half may be under way
                if (half && !warp_spin(&h_done[x], ns & 1)) ok = false;
                tc_fence_after();
#pragma unroll 1
                for (int i = 0; i < D; i += 16) {
                  uint32_t o[16];
                  tmem_ld16(tO + i, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
                  tmem_st16(tO + i, o);
                }
              }
            }
            l += sum;
          }
          tmem_st32(tS + half * 32, p);
          hand_over(half);
          arrive(half);
        }
        if (!ok) break;
      }
      if (!ok) break;
      // what needs no O comes before the wait for it (16 sequences of 100 to 1000
      // keys, D = 64: 40.4 -> 38.6 us)
      const float inv = l > 0.f ? 1.0f / l : l == 0.f ? 0.f : l;     // l is NaN: so is the row
      // 128 bytes of every row at a time pass through shared memory, swizzled as
      // a copy box is.  A warp whose 32 rows are whole heads of whole tokens, all
      // of this sequence, sends them with one bulk copy; others write them
      // eight lanes to a row (a thread's own row in 16-byte pieces would touch a
      // line with each).
      unsigned char* stage = smem + S::kOut + warp * 32 * 128;
      const int at = live ? token * a.Hq + g : -1;              // row's place after the tile's first
      const long long first = (long long)(it.row0 + x * t.tt) * a.Hq + it.head * G;
      const bool part = t.part_o != nullptr;
      if (part) {
        if (live) t.part_lse[(long long)it.split * a.T * a.Hq + first + at] = l > 0.f ? m + lg2(l) : l == 0.f ? -INFINITY : l;
      } else if (live && a.lse) {
        a.lse[first + at] = l > 0.f ? (m + lg2(l)) * 0.693147180559945f : l == 0.f ? -INFINITY : l;
      }
      const bool boxed = t.out_box && __all_sync(0xffffffffu, live);
      const int head0 = it.head * G + __shfl_sync(0xffffffffu, g, 0);
      const int token0 = it.row0 + x * t.tt + __shfl_sync(0xffffffffu, token, 0) + (part ? it.split * a.T : 0);
      auto put = [&](int unit, uint4 v) { *reinterpret_cast<uint4*>(stage + lane * 128 + ((unit ^ (lane & 7)) << 4)) = v; };
      auto write = [&](int column, int row_bytes) {             // of the output, bytes of its rows
        if (boxed) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) store_box(&tmO, stage, column, head0, token0);
          return;
        }
        __syncwarp();
        unsigned char* out =
            (part ? reinterpret_cast<unsigned char*>(t.part_o + (long long)it.split * a.T * a.Hq * D)
                  : reinterpret_cast<unsigned char*>(a.out)) +
            first * row_bytes + column * (row_bytes / D) + (lane & 7) * 16;
#pragma unroll 4
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + (lane >> 3), to = __shfl_sync(0xffffffffu, at, r);
          const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
          if (to >= 0) *reinterpret_cast<uint4*>(out + (long long)to * row_bytes) = v;
        }
        __syncwarp();
      };
      auto stage_free = [&]() {                                 // the bulk copies have read it
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
      };
      stage_free();
      if (n > 0 && !warp_spin(&o_full[x], no++ & 1)) { ok = false; break; }
      tc_fence_after();
      if (part) {
        if (n > 0)                                              // a part without keys is not read
#pragma unroll 1
          for (int i = 0; i < D; i += 32) {
            float v[32];
            tmem_ld32(tO + i, *reinterpret_cast<uint32_t(*)[32]>(v));
            tmem_wait_ld();
            if (i) stage_free();
#pragma unroll
            for (int u = 0; u < 8; ++u)
              put(u, make_uint4(__float_as_uint(v[4 * u] * inv), __float_as_uint(v[4 * u + 1] * inv),
                                __float_as_uint(v[4 * u + 2] * inv), __float_as_uint(v[4 * u + 3] * inv)));
            write(i, D * 4);
          }
      } else {
#pragma unroll 1
        for (int i = 0; i < D; i += 64) {
          float v[64];
          if (n > 0) {
            tmem_ld64(tO + i, v);
            tmem_wait_ld64(v);
          } else {
#pragma unroll
            for (int u = 0; u < 64; ++u) v[u] = 0.f;
          }
          uint4 w[8];
#pragma unroll
          for (int u = 0; u < 8; ++u)
            w[u] = make_uint4(pack2<kF16>(v[8 * u] * inv, v[8 * u + 1] * inv),
                              pack2<kF16>(v[8 * u + 2] * inv, v[8 * u + 3] * inv),
                              pack2<kF16>(v[8 * u + 4] * inv, v[8 * u + 5] * inv),
                              pack2<kF16>(v[8 * u + 6] * inv, v[8 * u + 7] * inv));
          if (i) stage_free();
#pragma unroll
          for (int u = 0; u < 8; ++u) put(u, w[u]);
          write(i, D * 2);
        }
      }
      tc_fence_before();
      if (*(volatile int*)abort_flag) { ok = false; break; }
    }
    if (!ok && lane == 0) atomicOr(abort_flag, 1);
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  tc_fence_before();
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) report(rep, blockIdx.x, (any ? kStatusBounds : 0) | (*abort_flag ? kStatusTimeout : 0));
  if (warp == kSoftWarps + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

// ------------------------------------------------------------------ host side
// 3-D map over the queries: {D, head, token}; box {64, G, tt}.
bool q_map(CUtensorMap* m, const AttnArgs& a, int tt) {
  const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
  const cuuint64_t strides[2] = {a.q.head * 2ull, a.q.tok * 2ull};
  const cuuint32_t box[3] = {64, (cuuint32_t)(a.Hq / a.Hkv), (cuuint32_t)tt};
  return encode(m, a.q.data, 3, dims, strides, box);
}

// 3-D map over the output, or over the parts in fp32: boxes of 32 rows x 128
// bytes, heads fastest.
int box_heads(const AttnArgs& a) {
  const int G = a.Hq / a.Hkv;
  return G < 32 ? G : G % 32 == 0 ? 32 : 33;
}
bool out_map(CUtensorMap* m, const AttnArgs& a, float* part_o, int splits) {
  const cuuint64_t size = part_o ? 4 : 2, heads = box_heads(a);
  const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.Hq, (cuuint64_t)a.T * (part_o ? splits : 1)};
  const cuuint64_t strides[2] = {a.D * size, (cuuint64_t)a.Hq * a.D * size};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / size), (cuuint32_t)heads, (cuuint32_t)(32 / heads)};
  return encode(m, part_o ? (const void*)part_o : a.out, 3, dims, strides, box,
                part_o ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
}

template <int D, bool kF16, bool kPaged>
cudaError_t launch(const TcAttnArgs& t, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                   const CUtensorMap& o, const Report& rep, int grid, cudaStream_t stream) {
  auto kern = attn_tc_kernel<D, kF16, kPaged>;
  constexpr size_t smem = Shape<D, kPaged>::kSmem;
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  kern<<<grid, kThreads, smem, stream>>>(q, k, v, o, t, rep);
  return cudaGetLastError();
}

}  // namespace

int tc_splits(const AttnArgs& a, int num_sms) {
  const TcPlan p = tc_plan(a);
  const long long units = (long long)p.slots * a.Hkv;
  const long long keys = a.prefix_table ? a.prefix_len : a.page_table ? (long long)a.table_pages << a.page_shift : a.Tk;
  const long long blocks = (keys + kKeys - 1) / kKeys;
  // (a shared prefix leaves SMs to the rows' own keys)
  long long s = (a.prefix_table ? num_sms - num_sms / kOwnShare : num_sms) / units;
  // (a prefix's parts are joined with the rows' own keys anyway)
  const int least = a.prefix_table ? 1 : kBlocksPerSplit;
  if (s > blocks / least) s = blocks / least;
  return s < 1 ? 1 : (int)s;
}

int tc_items(const AttnArgs& a, int splits) {
  const long long items = (long long)tc_plan(a).slots * a.Hkv * splits;
  return items < (1ll << 31) ? (int)items : -1;
}

cudaError_t launch_attn_tc(const AttnArgs& a, int splits, float* part_o, float* part_lse, const Report& shape,
                           cudaStream_t stream) {
  TcAttnArgs t{};
  t.a = a;
  const TcPlan p = tc_plan(a);
  t.tt = p.tt;
  t.slots = p.slots;
  t.splits = splits;
  t.G = a.Hq / a.Hkv;
  t.by_splits.set(splits);
  t.by_Hkv.set(a.Hkv);
  t.by_per.set(2 * p.tt);
  t.by_G.set(t.G);
  const int items = tc_items(a, splits);
  if (items < 0) return cudaErrorInvalidValue;
  t.box = a.page_table && (1 << a.page_shift) < kKeys ? 1 << a.page_shift : kKeys;
  t.c = a.scale * 1.4426950408889634f;
  // a scale of 0 (or so small that it would flush): so that a masked logit
  // stays one, and every other still counts as 0
  if (t.c < 1.2e-38f && t.c > -1.2e-38f) t.c = 1.2e-38f;
  t.hidden = t.c > 0 ? -INFINITY : INFINITY;
  t.part_o = part_o;
  t.part_lse = part_lse;
  t.arrivals = Arrivals(a.hold);
  const bool paged = a.page_table != nullptr;
  CUtensorMap q, k, v, o = {};
  if (!q_map(&q, a, t.tt)) return cudaErrorInvalidValue;
  // (parts of all splits are one tensor of splits * T tokens)
  t.out_box = 32 % box_heads(a) == 0 && (long long)a.T * splits < (1ll << 31);
  if (t.out_box && !out_map(&o, a, part_o, splits)) return cudaErrorInvalidValue;
  if (paged ? !pages_map(&k, a.k_cache, a, t.box) || !pages_map(&v, a.v_cache, a, t.box)
            : !rows_map(&k, a.k, a, a.Tk, a.Hkv, kKeys) || !rows_map(&v, a.v, a, a.Tk, a.Hkv, kKeys))
    return cudaErrorInvalidValue;
  Report rep = shape;
  rep.blocks[rep.set] = items;
#define TC_CASE(DD, F, P) \
  if (a.D == DD && (a.f16 != 0) == F && paged == P) return launch<DD, F, P>(t, q, k, v, o, rep, items, stream);
  TC_CASE(64, false, false)
  TC_CASE(64, false, true)
  TC_CASE(64, true, false)
  TC_CASE(64, true, true)
  TC_CASE(128, false, false)
  TC_CASE(128, false, true)
  TC_CASE(128, true, false)
  TC_CASE(128, true, true)
#undef TC_CASE
  return cudaErrorInvalidValue;
}

}  // namespace attn
}  // namespace moe
