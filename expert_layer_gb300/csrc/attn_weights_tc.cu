// Attention weight of every key (attn_weights.cu) for calls with many rows, on
// the tensor cores:
//   S' = K Q'                            tcgen05.mma, 128 keys x 128 rows, fp32 in tensor memory
//   w_j += sum_r exp2(c S'[j, r] - lse2[r])   lane = key, columns = rows
// so that a key's sum is one thread's: no exchange between lanes, and the rows'
// log-sums are the same for all of them (broadcast reads of shared memory).
//
// A unit is 256 keys of one sequence and head: two tiles of keys stay in shared
// memory while the rows pass by in tiles of 128 (tt tokens x G heads), each
// multiplied with both, for one warpgroup each (with one tile of keys a row tile
// would be read for 512 cycles of work, 64 bytes a cycle and SM from L2).  Blocks
// take equal ranges of the line of all units (attn_weights.cu).
// Measured: the last 64 rows of four prompts of 4000 to 16,000 keys (32 query and 4
// key-value heads of 128) 31.8 us, on mma.sync 111.  Its exponentials (32 a cycle
// and SM) are 6.5 us of that, its products (2 x 512 cycles for each row tile, D =
// 128) 7, the start 5.5; neither pipe is its bound (tensor pipe 19% busy, issue slots
// 21%).  A warp of the sums loads S and then sums it, an entry is read when its unit
// ends, and 512 units are 3.4 uneven rounds of 152 SMs.
#include "attn.h"
#include "attn_ptx.cuh"
#include "weights_line.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kRows = 128;              // of a row tile
constexpr int kKeys = 256;              // of a unit: two tiles
constexpr int kItems = 4;               // ring of units
constexpr int kRowStages = 2;           // ring of the rows' log-sums
constexpr int kSumWarps = 8;
constexpr int kThreads = (kSumWarps + 4) * 32;
constexpr uint32_t kTmemCols = 512;
constexpr int kUnitTiles = 1;           // cost of a unit's keys, in row tiles

template <int D>
struct Shape {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalfBytes = kRows * 128;               // a 128-byte wide column of a row tile
  static constexpr int kQTile = kHalves * kHalfBytes;
  static constexpr int kGroup = kHalves * 1024;                // 8 keys (pages_map)
  static constexpr int kKTile = 128 * D * 2;
  static constexpr int kQStages = D == 128 ? 3 : 6;
  static constexpr int kQ = 4 * kKTile;                        // two units' keys come first
  static constexpr int kRowsAt = kQ + kQStages * kQTile;       // [stage]: 128 offsets, 128 limits
  static constexpr int kBars = kRowsAt + kRowStages * 1024;
  static constexpr size_t kSmem = kBars + 768;
};
static_assert(Shape<128>::kSmem <= 232448 && Shape<64>::kSmem <= 232448, "227 KB a block");

struct Unit {
  int s;               // -1: no more
  int q0, n, len, head, k0;
  int t0, tiles;       // first row tile that sees a key, and their number
};
struct RowMeta {
  int whole;           // each of the tt G rows is one of the sequence's, with keys
  int least;           // the first key that some row does not see, less one
};

template <int D, bool kF16>
__global__ void __launch_bounds__(kThreads, 1)
    attn_weights_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const WeightArgs a, const Report rep, const int tt, const int box) {
  using S = Shape<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t* k_empty = k_full + 2;
  uint64_t* q_full = k_empty + 2;
  uint64_t* q_empty = q_full + S::kQStages;
  uint64_t* r_full = q_empty + S::kQStages;
  uint64_t* r_empty = r_full + kRowStages;
  uint64_t* s_full = r_empty + kRowStages;
  uint64_t* s_empty = s_full + 2;
  uint64_t* it_full = s_empty + 2;
  uint64_t* it_empty = it_full + kItems;
  uint64_t* drain = it_empty + kItems;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  Unit* ring = reinterpret_cast<Unit*>(tmem_slot + 2);
  RowMeta* meta = reinterpret_cast<RowMeta*>(ring + kItems);
  LineStart<kThreads>& start = *reinterpret_cast<LineStart<kThreads>*>(smem + S::kBars + 512);
  static_assert(sizeof(start) <= 256, "start of the block's range");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.Hq / a.Hkv;
  bool bad = false;
  if (threadIdx.x == 0) {
    prefetch_map(&tmQ);
    prefetch_map(&tmK);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1 + (a.hold == kHoldKeys));
      mbar_init(&k_empty[i], 1);
      mbar_init(&s_full[i], 1 + (a.hold == kHoldS));
      mbar_init(&s_empty[i], kSumWarps);
    }
    for (int i = 0; i < S::kQStages; ++i) {
      mbar_init(&q_full[i], 1 + (a.hold == kHoldQuery));
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < kRowStages; ++i) {
      mbar_init(&r_full[i], 1);
      mbar_init(&r_empty[i], kSumWarps);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], kSumWarps + 2);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == kSumWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // rows of a tile beyond tt * G are never loaded: zeros
  if (tt * G < kRows)
    for (int i = threadIdx.x; i < S::kQStages * S::kQTile / 16; i += kThreads)
      reinterpret_cast<uint4*>(smem + S::kQ)[i] = make_uint4(0, 0, 0, 0);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  // a unit's cost and a sequence's units (of all heads)
  auto cost = [&](const Seq& v) { return (v.n + tt - 1) / tt + kUnitTiles; };
  auto units = [&](const Seq& v) { return v.n ? (v.len + kKeys - 1) / kKeys : 0; };
  find_start(a, start, 1, [&](const Seq& v) { return (long long)units(v) * a.Hkv * cost(v); }, bad);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto gave_up = [&]() { return *(volatile int*)abort_flag != 0; };

  if (warp == kSumWarps) {
    // ------------------------------------------------------------ units, loads
    uint32_t nk = 0, nq = 0, ni = 0;
    bool ok = true;
    const long long begin = start.begin(blockIdx.x), end = start.begin(blockIdx.x + 1);
    int s = start.seq[0];
    long long at = start.at[0], u = 0;
    Seq v{};
    if (s >= 0) {
      v = seq_of(a, s, bad);
      u = (begin - at + cost(v) - 1) / cost(v);    // a unit belongs to the block whose range holds its first place
    }
    while (ok) {
      Unit it;
      it.s = -1;
      if (s >= 0) {
        while (u >= (long long)units(v) * a.Hkv) {
          at += (long long)units(v) * a.Hkv * cost(v);
          if (++s >= a.n_seq) break;
          v = seq_of(a, s, bad);
          u = 0;
        }
        if (s < a.n_seq && at + u * cost(v) < end) {
          it = Unit{s, v.q0, v.n, v.len, (int)(u / units(v)), 0, 0, (v.n + tt - 1) / tt};
          it.k0 = (int)(u - (long long)it.head * units(v)) * kKeys;
          it.t0 = a.causal ? max(0, it.k0 - (v.len - v.n)) / tt : 0;
          ++u;
          if (it.t0 >= it.tiles) continue;         // no row sees any of its keys
        }
      }
      // page of this lane's box, under way while the ring is waited for
      const int nbox = it.s < 0 ? 0 : (min(kKeys, it.len - it.k0) + box - 1) / box;
      int page = 0;
      if (lane < nbox) page = a.page_table[(long long)it.s * a.table_pages + ((it.k0 + lane * box) >> a.page_shift)];
      const int slot = ni % kItems;
      ok = warp_spin(&it_empty[slot], ((ni / kItems) & 1) ^ 1);
      if (!ok) break;
      if (lane == 0) {
        ring[slot] = it;
        mbar_arrive(&it_full[slot]);
      }
      ++ni;
      if (it.s < 0) break;
      const int kb = nk & 1;
      ok = warp_spin(&k_empty[kb], ((nk >> 1) & 1) ^ 1);
      if (!ok) break;
      if ((unsigned)page >= (unsigned)a.pages) bad = true, page = 0;
      if (lane == 0) mbar_expect_tx(&k_full[kb], (uint32_t)(nbox * box * D * 2));
      __syncwarp();
      if (lane < nbox)
        tma_load_5d(smem + kb * 2 * S::kKTile + lane * (box / 8) * S::kGroup, &tmK, 0, 0, 0,
                    ((it.k0 + lane * box) & ((1 << a.page_shift) - 1)) / 8, page * a.Hkv + it.head, &k_full[kb]);
      ++nk;
      for (int t = it.t0; t < it.tiles; ++t) {
        const int st = nq % S::kQStages;
        ok = warp_spin(&q_empty[st], ((nq / S::kQStages) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          mbar_expect_tx(&q_full[st], (uint32_t)(S::kHalves * G * tt * 128));
          for (int hh = 0; hh < S::kHalves; ++hh)
            tma_load_3d(smem + S::kQ + st * S::kQTile + hh * S::kHalfBytes, &tmQ, hh * 64, it.head * G, it.q0 + t * tt,
                        &q_full[st]);
        }
        ++nq;
      }
      if (gave_up()) ok = false;
    }
    if (lane == 0) {
      if (!ok) atomicOr(abort_flag, 1);
      // the loads issued land before the block exits
      for (uint32_t i = nk > 2 ? nk - 2 : 0; i < nk; ++i) spin_wait(&k_full[i & 1], (i >> 1) & 1);
      for (uint32_t i = nq > (uint32_t)S::kQStages ? nq - S::kQStages : 0; i < nq; ++i)
        spin_wait(&q_full[i % S::kQStages], (i / S::kQStages) & 1);
    }
    __syncwarp();
  } else if (warp == kSumWarps + 1) {
    // ------------------------------------------------------------ products
    constexpr uint32_t kId = (1u << 4) | ((kF16 ? 0u : 1u) << 7) | ((kF16 ? 0u : 1u) << 10) |
                             ((uint32_t)(kRows >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
    uint32_t nk = 0, nq = 0, ni = 0;
    bool ok = true;
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) umma_commit(bar);
      __syncwarp();
    };
    while (ok) {
      const int slot = ni % kItems;
      ok = warp_spin(&it_full[slot], (ni / kItems) & 1);
      if (!ok) break;
      const int s = __reduce_max_sync(0xffffffffu, ring[slot].s);
      const int count = __reduce_max_sync(0xffffffffu, ring[slot].tiles - ring[slot].t0);
      const int two = __reduce_max_sync(0xffffffffu, ring[slot].k0 + 128 < ring[slot].len ? 1 : 0);
      if (lane == 0) mbar_arrive(&it_empty[slot]);
      __syncwarp();
      ++ni;
      if (s < 0) break;
      const int kb = __reduce_max_sync(0xffffffffu, nk & 1);
      ok = warp_spin(&k_full[kb], (nk >> 1) & 1);
      ++nk;
#pragma unroll 1
      for (int t = 0; t < count && ok; ++t, ++nq) {
        const int st = __reduce_max_sync(0xffffffffu, nq % S::kQStages), p = nq & 1;
        ok = warp_spin(&q_full[st], (nq / S::kQStages) & 1) && warp_spin(&s_empty[p], ((nq >> 1) & 1) ^ 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t dq = umma_desc(smem_u32(smem) + S::kQ + st * S::kQTile);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (x && !two) continue;
            const uint64_t dk = umma_desc_k(smem_u32(smem) + (kb * 2 + x) * S::kKTile, S::kGroup);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_bf16_id(p * 256 + x * 128, dk + (((kk / 4) * 1024 + (kk % 4) * 32) >> 4),
                           dq + (((kk / 4) * S::kHalfBytes + (kk % 4) * 32) >> 4), kId, kk ? 1u : 0u);
          }
          umma_commit(&s_full[p]);
          umma_commit(&q_empty[st]);
        }
        __syncwarp();
      }
      if (!ok) break;
      commit(&k_empty[kb]);
      if (gave_up()) ok = false;
    }
    // the MMAs issued finish before their memory is freed, whoever gives up
    if (!ok && lane == 0) atomicOr(abort_flag, 1);
    commit(drain);
    if (lane == 0) spin_wait(drain, 0);
    __syncwarp();
  } else if (warp == kSumWarps + 2) {
    // ------------------------------------------------------------ the rows' log-sums and limits
    uint32_t nr = 0, ni = 0;
    bool ok = true;
    while (ok) {
      const int slot = ni % kItems;
      ok = warp_spin(&it_full[slot], (ni / kItems) & 1);
      if (!ok) break;
      const Unit it = ring[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&it_empty[slot]);
      ++ni;
      if (it.s < 0) break;
      for (int t = it.t0; t < it.tiles; ++t, ++nr) {
        float off[4];
        int lim[4], least = 0x7fffffff;
        bool whole = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 4 * lane + i, in = a.by_G.of(r), token = t * tt + in;
          const bool there = in < tt && token < it.n;
          const float l =
              there ? a.lse[(long long)(it.q0 + token) * a.Hq + it.head * G + r - in * G] : -INFINITY;
          // a row without keys, and one that is not there, give nothing
          off[i] = l == -INFINITY ? -INFINITY : -l * 1.4426950408889634f;
          lim[i] = a.causal ? min(token + it.len - it.n, it.len - 1) : it.len - 1;
          if (in < tt) {
            whole &= off[i] != -INFINITY;
            least = min(least, lim[i]);
          }
        }
        const int rs = nr % kRowStages;
        ok = warp_spin(&r_empty[rs], ((nr / kRowStages) & 1) ^ 1);
        if (!ok) break;
        float* at = reinterpret_cast<float*>(smem + S::kRowsAt + rs * 1024);
        *reinterpret_cast<float4*>(at + 4 * lane) = make_float4(off[0], off[1], off[2], off[3]);
        *reinterpret_cast<int4*>(at + kRows + 4 * lane) = make_int4(lim[0], lim[1], lim[2], lim[3]);
        whole = __all_sync(0xffffffffu, whole);
        least = __reduce_min_sync(0xffffffffu, least);
        if (lane == 0) meta[rs] = RowMeta{whole, least};
        __syncwarp();
        if (lane == 0) mbar_arrive(&r_full[rs]);
      }
      if (gave_up()) ok = false;
    }
    if (!ok && lane == 0) atomicOr(abort_flag, 1);
    __syncwarp();
  } else if (warp < kSumWarps) {
    // ------------------------------------------------------------ sums
    const int x = warp >> 2;                                   // tile of keys
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t nr = 0, ni = 0;
    bool ok = true;
    const uint64_t c2 = pair(a.c, a.c);
    while (ok) {
      const int slot = ni % kItems;
      ok = warp_spin(&it_full[slot], (ni / kItems) & 1);
      if (!ok) break;
      const Unit it = ring[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&it_empty[slot]);
      ++ni;
      if (it.s < 0) break;
      const int first = it.k0 + x * 128, key = first + (warp & 3) * 32 + lane;
      const bool active = first < it.len;
      uint64_t sum[2] = {0, 0};
#pragma unroll 1
      for (int t = it.t0; t < it.tiles; ++t, ++nr) {
        const int p = nr & 1, rs = nr % kRowStages;
        ok = warp_spin(&r_full[rs], (nr / kRowStages) & 1) && warp_spin(&s_full[p], (nr >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const RowMeta m = meta[rs];
        const float4* off = reinterpret_cast<const float4*>(smem + S::kRowsAt + rs * 1024);
        const int4* lim = reinterpret_cast<const int4*>(off + kRows / 4);
        const int parts = active ? (min(tt, it.n - t * tt) * G + 31) / 32 : 0;      // of 32 rows
        // parts without a masked row; the rows from tt G on, which are zeros, count as
        // masked (times a key's infinity they are NaN)
        const int plain = m.whole && m.least >= first + 127 ? tt * G / 32 : 0;
#pragma unroll 1
        for (int part = 0; part < parts; ++part) {
          float s[32];
          tmem_ld32(tmem + lanes + p * 256 + x * 128 + part * 32, *reinterpret_cast<uint32_t(*)[32]>(s));
          tmem_wait_ld();
          if (part + 1 == parts) {                 // the next product may overwrite it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[p]);
          }
          if (part < plain) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float4 o = off[part * 8 + k];
              const uint64_t y0 = fma2(pair(s[4 * k], s[4 * k + 1]), c2, pair(o.x, o.y));
              const uint64_t y1 = fma2(pair(s[4 * k + 2], s[4 * k + 3]), c2, pair(o.z, o.w));
              sum[0] = add2(sum[0], pair(ex2(lo(y0)), ex2(hi(y0))));
              sum[1] = add2(sum[1], pair(ex2(lo(y1)), ex2(hi(y1))));
            }
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float4 o = off[part * 8 + k];
              const int4 l = lim[part * 8 + k];
              // (a row that another sequence has may hold anything)
              auto one = [&](float v, float o, int l) {
                return o == -INFINITY || key > l ? 0.f : ex2(fmaf(v, a.c, o));
              };
              sum[0] = add2(sum[0], pair(one(s[4 * k], o.x, l.x), one(s[4 * k + 1], o.y, l.y)));
              sum[1] = add2(sum[1], pair(one(s[4 * k + 2], o.z, l.z), one(s[4 * k + 3], o.w, l.w)));
            }
          }
        }
        __syncwarp();
        if (lane == 0) {
          if (parts == 0) mbar_arrive(&s_empty[p]);
          mbar_arrive(&r_empty[rs]);
        }
      }
      if (!ok) break;
      sum[0] = add2(sum[0], sum[1]);
      if (active && key < it.len) {
        float* w = a.weights + ((long long)it.s * a.Hkv + it.head) * a.capacity + key;
        *w += lo(sum[0]) + hi(sum[0]);
      }
      if (gave_up()) ok = false;
    }
    if (!ok && lane == 0) atomicOr(abort_flag, 1);
    __syncwarp();
  }
  tc_fence_before();
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) report(rep, blockIdx.x, (any ? kStatusBounds : 0) | (*abort_flag ? kStatusTimeout : 0));
  if (warp == kSumWarps + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

template <int D, bool kF16>
cudaError_t launch(const WeightArgs& a, const CUtensorMap& q, const CUtensorMap& k, const Report& rep, int tt, int box,
                   int grid, cudaStream_t stream) {
  auto kern = attn_weights_tc_kernel<D, kF16>;
  constexpr size_t smem = Shape<D>::kSmem;
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  kern<<<grid, kThreads, smem, stream>>>(q, k, a, rep, tt, box);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_weights_tc(const WeightArgs& a, void* ws, int num_sms, cudaStream_t stream) {
  const Report rep{ws, 0, {num_sms, 0}};
  const int tt = kRows / (a.Hq / a.Hkv), box = 1 << a.page_shift < 128 ? 1 << a.page_shift : 128;
  CUtensorMap q, k;
  if (!q_map(&q, a.q, a.T, a.Hq, a.Hkv, a.D, tt) ||
      !pages_map(&k, a.k_cache, a.D, a.page_shift, a.pages, a.Hkv, box))
    return cudaErrorInvalidValue;
  if (a.D == 64)
    return a.f16 ? launch<64, true>(a, q, k, rep, tt, box, num_sms, stream)
                 : launch<64, false>(a, q, k, rep, tt, box, num_sms, stream);
  return a.f16 ? launch<128, true>(a, q, k, rep, tt, box, num_sms, stream)
               : launch<128, false>(a, q, k, rep, tt, box, num_sms, stream);
}

}  // namespace attn
}  // namespace moe
