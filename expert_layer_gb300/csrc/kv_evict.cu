// Eviction from the paged cache by accumulated weight: of a sequence's n keys
// each head keeps the first `first`, the last `last` and, of those between, the
// ones of largest weight, `budget` in all (ties: the first key; a NaN counts as
// the smallest).  What is kept moves to other pages in its order.
//
// Two kernels.  The first takes a (sequence, head) per block: the rank that the
// last kept key's weight has, two bits at a time from the top, counted over keys
// in registers (more than 16,384: three passes with a histogram of 11 bits, 11
// and 10), then one pass in key order that gives every kept key its place.  The
// second copies the rows, any order, with the places from the first.  Copying to
// other pages rather than within them leaves every row free of the others', and
// pages that sequences share as they were.
// Bound: HBM for the copy (8 D bytes a kept key and head), latency for the first:
// 64 sequences, 4 heads of 128, 16,384 keys at most, 1024 kept: 60 us, the copy 34
// of them; the first kernel's time is the chain of a long item, up to 16 counts
// with a barrier each (long and short items paired on the SMs: equal).  One kernel
// for both: 90 us, rows wait for their search.
#include "attn.h"
#include "attn_ptx.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kBins = 2048;
// Unsigned in the order of the weights
__device__ __forceinline__ uint32_t rank_of(float w) {
  if (!(w == w)) return 0;
  const uint32_t b = __float_as_uint(w + 0.0f);                // -0 is 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Keys of a sequence; none (and `bad`) where its length is out of range
__device__ __forceinline__ int keys_of(const EvictArgs& a, int s, bool& bad) {
  int n = a.kv_lens[s];
  if (n < 0 || n > a.capacity || n > ((long long)a.table_pages << a.page_shift)) bad = true, n = 0;
  return n;
}

// Sum over the threads before this one, and over all
template <int kWarps>
__device__ __forceinline__ int block_scan(int v, int* warps, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += x;
  }
  __syncthreads();                          // `warps` is free
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  int w = warps[lane & (kWarps - 1)], sum = w;
#pragma unroll
  for (int d = 1; d < kWarps; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, sum, d, kWarps);
    if ((lane & (kWarps - 1)) >= d) sum += x;
  }
  total = __shfl_sync(0xffffffffu, sum, kWarps - 1);
  return incl - v + __shfl_sync(0xffffffffu, sum - w, warp);
}

// kEach: keys of a thread, where they are counted
template <int kThreads, int kEach>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) evict_select_kernel(const EvictArgs a, const Report rep) {
  constexpr int kWarps = kThreads / 32, kTile = kThreads * kEach;
  extern __shared__ float keys[];          // weights of a tile of keys
  __shared__ int2 totals[kWarps];
  constexpr int kOwn = kBins / kThreads;    // bins of a thread, spread over the banks as the keys are
  auto bin = [](int b) { return b + b / kOwn; };
  __shared__ int bins[kBins + kThreads];
  __shared__ int warps[kWarps];
  __shared__ int found[2];                  // a digit, and the keys above it
  __shared__ __align__(16) int2 counts[2][kWarps];
  bool bad = false;
  pdl_trigger();                            // the copy kernel waits for this grid's end
  for (int item = blockIdx.x; item < a.n_seq * a.Hkv; item += gridDim.x) {
    const int s = a.by_Hkv.of(item), head = item - s * a.Hkv;
    const int n = keys_of(a, s, bad);
    const float* w = a.weights + (long long)item * a.capacity;
    float* to = a.new_weights + (long long)item * a.budget;
    int32_t* kept = a.kept + (long long)item * a.budget;
    const int m = min(n, a.budget);
    for (int i = m + threadIdx.x; i < a.budget; i += kThreads) {
      to[i] = 0.f;
      kept[i] = -1;
    }
    if (n <= a.budget) {
      for (int i = threadIdx.x; i < n; i += kThreads) {
        to[i] = w[i];
        kept[i] = i;
      }
      continue;
    }
    const int lo = a.first, hi = n - a.last;
    int need = a.budget - a.first - a.last; // of the keys lo .. hi - 1, fewer than there are
    // Up to a tile of keys is read once, more are read anew each time.  Ranks in
    // registers for the search, which takes them several times; the places are
    // given from shared memory, in a small loop (code that an item runs once comes
    // from L2 as it runs, ~100 cycles for eight instructions).
    const bool single = n <= kTile;
    uint32_t rank[kEach];                   // 0 for keys that are always kept
    auto load = [&](int i0) {
      float x[kEach];
#pragma unroll
      for (int j = 0; j < kEach; ++j) x[j] = w[min(i0 + j * kThreads + (int)threadIdx.x, n - 1)];
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int i = j * kThreads + (int)threadIdx.x;
        rank[j] = i0 + i >= lo && i0 + i < hi ? rank_of(x[j]) : 0;
        keys[i] = x[j];
      }
    };
    __syncthreads();                        // those of the item before have been used
    if (single) load(0);
    // --- the rank that the last key kept has, and how many of those that have it are
    uint32_t prefix = 0, mask = 0;
    if (need > 0 && single) {
      // two bits at a time: the largest rank that `need` keys reach.  (A histogram
      // of digits in its place: the counts of a heavy tail meet in a few bins.
      // Whole calls, 64 sequences of 4 heads and up to 16,384 keys 69 -> 66 us, 8
      // sequences of 2 heads and up to 700 keys 7.6 -> 6.4.)
      mask = ~0u;
      int above = 0, from = n, base = 0;    // keys beyond the range that is left, and from its start on
      // Once the range holds few keys they go to a list, a few to a thread: a step
      // over 17,000 keys of an SM takes 1.5 us (66 -> 62 us).  Not for tiles of 16 to
      // a thread, whose steps are short (6.4 -> 6.8).
      constexpr int kList = 2;
      constexpr bool kLists = kEach > 16;
      bool listed = false;
      uint32_t few[kList] = {};
      uint32_t* list = reinterpret_cast<uint32_t*>(bins);
      static_assert(kList * kThreads <= kBins + kThreads, "the list takes the place of the bins");
#pragma unroll 1
      for (int shift = 30; shift >= 0; shift -= 2) {
        const uint32_t c1 = prefix | 1u << shift, c2 = prefix | 2u << shift, c3 = prefix | 3u << shift;
        int n1 = 0, n2 = 0, n3 = 0;         // up to 2^14 of each
        auto count = [&](uint32_t r) {
          asm("{\n .reg .pred p, q, r;\n setp.ge.u32 p, %3, %4;\n setp.ge.u32 q, %3, %5;\n setp.ge.u32 r, %3, %6;\n"
              " @p add.s32 %0, %0, 1;\n @q add.s32 %1, %1, 1;\n @r add.s32 %2, %2, 1;\n}\n"
              : "+r"(n1), "+r"(n2), "+r"(n3)
              : "r"(r), "r"(c1), "r"(c2), "r"(c3));
        };
        if (kLists && !listed && from - above <= kList * kThreads && n > 2 * kList * kThreads) {
          listed = true;
          base = above;
          const uint32_t width = 4u << shift;          // of the range (0: all)
          const uint32_t least = max(prefix, 1u);      // rank 0: no key, or never counted
          int own = 0, all;
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            if (j % 8 == 0 && j * kThreads >= n) break;
            own += rank[j] >= least && rank[j] - prefix < width;
          }
          int to_list = block_scan<kWarps>(own, warps, all);
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            if (j % 8 == 0 && j * kThreads >= n) break;
            if (rank[j] >= least && rank[j] - prefix < width) {
              if (to_list < kList * kThreads) list[to_list] = rank[j];
              ++to_list;
            }
          }
          __syncthreads();
#pragma unroll
          for (int j = 0; j < kList; ++j) {
            const int i = j * kThreads + (int)threadIdx.x;
            few[j] = i < all ? list[i] : 0;
          }
          __syncthreads();
        }
        if (kLists && listed) {
#pragma unroll
          for (int j = 0; j < kList; ++j) count(few[j]);
        } else {
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            if (j % 8 == 0 && j * kThreads >= n) break;
            count(rank[j]);
          }
        }
        int n12 = __reduce_add_sync(0xffffffffu, n1 | n2 << 16);
        n3 = __reduce_add_sync(0xffffffffu, n3);
        int2* all = counts[(shift >> 1) & 1];
        if ((threadIdx.x & 31) == 0) all[threadIdx.x >> 5] = make_int2(n12, n3);
        __syncthreads();
        n12 = n3 = 0;
#pragma unroll
        for (int k = 0; k < kWarps; k += 2) {
          const int4 v = *reinterpret_cast<const int4*>(&all[k]);
          n12 += v.x + v.z;
          n3 += v.y + v.w;
        }
        n1 = n12 & 0xffff, n2 = n12 >> 16;
        if (kLists && listed) n1 += base, n2 += base, n3 += base;
        const int digit = n3 >= need ? 3 : n2 >= need ? 2 : n1 >= need ? 1 : 0;
        prefix |= (uint32_t)digit << shift;
        above = digit == 3 ? above : digit == 2 ? n3 : digit == 1 ? n2 : n1;
        if (digit) from = digit == 3 ? n3 : digit == 2 ? n2 : n1;
        if (digit && from == need) {     // those from here on, and no other
          prefix -= 1;
          above = need;
          break;
        }
      }
      need -= above;
    } else if (need > 0) {
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 1024 : 2048;
        for (int i = threadIdx.x; i < kBins + kThreads; i += kThreads) bins[i] = 0;
        __syncthreads();
        for (int i0 = 0; i0 < hi; i0 += kTile) {
          load(i0);                         // (each thread counts those that it loads)
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            const int i = i0 + j * kThreads + (int)threadIdx.x;
            if (i >= lo && i < hi && (rank[j] & mask) == prefix)
              atomicAdd(&bins[bin((rank[j] >> shift) & (width - 1))], 1);
          }
        }
        __syncthreads();
        // from the largest digit down: a thread has the next kOwn of them
        int own = 0, total;
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          const int b = width - 1 - ((int)threadIdx.x * kOwn + j);
          own += b >= 0 ? bins[bin(b)] : 0;
        }
        int above = block_scan<kWarps>(own, warps, total);
        if (above < need && above + own >= need)
          for (int j = 0; j < kOwn; ++j) {
            const int b = width - 1 - ((int)threadIdx.x * kOwn + j);
            if (above + bins[bin(b)] >= need) {
              found[0] = b;
              found[1] = above;
              break;
            }
            above += bins[bin(b)];
          }
        __syncthreads();
        prefix |= (uint32_t)found[0] << shift;
        mask |= (uint32_t)(width - 1) << shift;
        need -= found[1];                   // of those that share the digits so far
        __syncthreads();
      }
    }
    // --- places, in key order; `need` keys of the rank `prefix` are kept, the
    // first ones.  A warp takes consecutive rows of 32 keys, lane j keeps the bits
    // of its row j.
    static_assert(kEach <= 32, "a lane for each row of a warp");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int at = 0, ties = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kTile) {
      if (!single) {
        __syncthreads();                    // those of the tile before have been used
        load(i0);
      }
      __syncthreads();
      const int rows = (min(kTile, n - i0) + 32 * kWarps - 1) / (32 * kWarps), row0 = warp * rows;
      uint32_t kept_of = 0, equal = 0;
#pragma unroll 4
      for (int j = 0; j < rows; ++j) {
        const int i = (row0 + j) * 32 + lane;
        const uint32_t r = rank_of(keys[i]);
        const bool there = i0 + i < n, middle = there && i0 + i >= lo && i0 + i < hi;
        const uint32_t gt = __ballot_sync(0xffffffffu, middle ? mask && r > prefix : there);
        const uint32_t eq = __ballot_sync(0xffffffffu, middle && mask && r == prefix);
        if (lane == j) kept_of = gt, equal = eq;
      }
      auto before = [&](int v) {            // sum over the lanes before this one
        int sum = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, sum, d);
          if (lane >= d) sum += o;
        }
        return sum - v;
      };
      const int larger = __reduce_add_sync(0xffffffffu, __popc(kept_of)), same = __popc(equal);
      const int same_before = before(same);
      if (lane == 31) totals[warp] = make_int2(larger, same_before + same);
      __syncthreads();
      const int2 t = lane < kWarps ? totals[lane] : make_int2(0, 0);         // of warp `lane`
      const int t_ties = ties + before(t.y);
      const int t_kept = t.x + max(0, min(t.y, need - t_ties)), t_at = at + before(t_kept);
      ties += __reduce_add_sync(0xffffffffu, t.y);
      at += __reduce_add_sync(0xffffffffu, t_kept);
      const int mine = __shfl_sync(0xffffffffu, t_ties, warp) + same_before;
      for (int extra = same - max(0, need - mine); extra > 0 && equal; --extra) equal &= ~(0x80000000u >> __clz(equal));
      kept_of |= equal;
      const int first = __shfl_sync(0xffffffffu, t_at, warp) + before(__popc(kept_of));
#pragma unroll 1
      for (uint32_t todo = __ballot_sync(0xffffffffu, kept_of != 0); todo; todo &= todo - 1) {
        const int j = __ffs(todo) - 1, i = (row0 + j) * 32 + lane;
        const uint32_t row = __shfl_sync(0xffffffffu, kept_of, j);
        const int place = __shfl_sync(0xffffffffu, first, j) + __popc(row & ((1u << lane) - 1));
        if ((row >> lane) & 1) {
          to[place] = keys[i];
          kept[place] = i0 + i;
        }
      }
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) report(rep, blockIdx.x, any ? kStatusBounds : 0);
}

// Rows of the kept keys, 16 bytes of K and of V per thread.  A last block writes the
// new lengths, when every head's selection has read the old ones: they may be one array.
constexpr int kCopyThreads = 256;
template <int D>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictArgs a, const Report rep) {
  constexpr int kLanes = D / 8;
  pdl_wait();
  bool bad = false;
  if (blockIdx.x == gridDim.x - 1) {                 // (what is out of range has been reported)
    for (int s = threadIdx.x; s < a.n_seq; s += kCopyThreads) a.new_lens[s] = min(keys_of(a, s, bad), a.budget);
    return;
  }
  const int lane = threadIdx.x % kLanes;
  const long long rows = (long long)a.n_seq * a.Hkv * a.budget;
  const int in_page = (1 << a.page_shift) - 1;
  for (long long r = ((long long)blockIdx.x * kCopyThreads + threadIdx.x) / kLanes; r < rows;
       r += (long long)(gridDim.x - 1) * (kCopyThreads / kLanes)) {
    const int key = a.kept[r];
    if (key < 0) continue;
    const int item = r >> 31 ? (int)(r / a.budget) : a.by_budget.of((int)r), place = (int)(r - (long long)item * a.budget);
    const int s = a.by_Hkv.of(item), head = item - s * a.Hkv;
    const int from = a.page_table[(long long)s * a.table_pages + (key >> a.page_shift)];
    const int to = a.out_table[(long long)s * a.out_pages + (place >> a.page_shift)];
    if ((unsigned)from >= (unsigned)a.pages || (unsigned)to >= (unsigned)a.pages) {
      bad = true;
      continue;
    }
    const long long src = ((((long long)from * a.Hkv + head) << a.page_shift) + (key & in_page)) * D + lane * 8;
    const long long dst = ((((long long)to * a.Hkv + head) << a.page_shift) + (place & in_page)) * D + lane * 8;
    const uint4 k = *reinterpret_cast<const uint4*>(a.k_cache + src);
    const uint4 v = *reinterpret_cast<const uint4*>(a.v_cache + src);
    *reinterpret_cast<uint4*>(a.k_cache + dst) = k;
    *reinterpret_cast<uint4*>(a.v_cache + dst) = v;
  }
  // the first kernel's words are complete: what was found here joins one of them
  if (__syncthreads_or(bad) && threadIdx.x == 0)
    atomicOr(reinterpret_cast<int*>(reinterpret_cast<char*>(rep.ws) + sizeof(Header)) + blockIdx.x % rep.blocks[0],
             kStatusBounds);
}

template <int kThreads, int kEach>
cudaError_t select(const EvictArgs& a, const Report& rep, int grid, cudaStream_t stream) {
  auto kern = evict_select_kernel<kThreads, kEach>;
  constexpr int smem = kThreads * kEach * 4;
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  kern<<<grid, kThreads, smem, stream>>>(a, rep);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& a, void* ws, int num_sms, cudaStream_t stream) {
  const int items = a.n_seq * a.Hkv, grid = items < kFlagsFirst ? items : kFlagsFirst;
  const Report rep{ws, 0, {grid, 0}};
  // threads by the most keys there can be: with 512 for all, 8 sequences of up to
  // 700 keys 7.6 us, with 128 6.4; a block holds at most 32 keys a thread in registers
  const cudaError_t err = a.capacity <= 2048   ? select<128, 16>(a, rep, grid, stream)
                          : a.capacity <= 4096 ? select<256, 16>(a, rep, grid, stream)
                                               : select<512, 32>(a, rep, grid, stream);
  if (err != cudaSuccess) return err;
  const long long rows = (long long)items * a.budget, blocks = (rows * (a.D / 8) + kCopyThreads - 1) / kCopyThreads;
  const long long most = 16ll * num_sms;
  auto kern = a.D == 64 ? evict_copy_kernel<64> : evict_copy_kernel<128>;
  return launch_pdl(kern, dim3((unsigned)(blocks < most ? blocks : most) + 1), dim3(kCopyThreads), 0, stream, a, rep);
}

}  // namespace attn
}  // namespace moe
