// Eviction from the paged cache by accumulated weight: of a sequence's n keys
// each head keeps the first `first`, the last `last` and, of those between, the
// ones of largest weight, `budget` in all (ties: the first key; a NaN counts as
// the smallest).  What is kept moves to other pages in its order.
//
// Two kernels.  The first takes a (sequence, head) per block: the weight that the
// last kept key has, digit by digit from the top (a radix select: three passes
// over the weights with a histogram of 2048, 2048 and 1024 bins), then one pass
// in key order that gives every kept key its place.  The second copies the rows,
// any order, with the places from the first.  Copying to other pages rather than
// within them leaves every row free of the others', and pages that sequences
// share as they were.
// Bound: HBM for the copy (8 D bytes a kept key and head), latency for the first.
#include "attn.h"
#include "attn_ptx.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kEach = 4;                    // consecutive keys of a thread
constexpr int kTile = kThreads * kEach;

// Unsigned in the order of the weights
__device__ __forceinline__ uint32_t rank_of(float w) {
  if (!(w == w)) return 0;
  const uint32_t b = __float_as_uint(w + 0.0f);                // -0 is 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Sum over the threads before this one, and over all
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

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictArgs a, const Report rep) {
  __shared__ int bins[kBins];
  __shared__ int warps[kWarps];
  __shared__ int found[2];                  // a digit, and the keys above it
  bool bad = false;
  pdl_trigger();                            // the copy kernel waits for this grid's end
  for (int item = blockIdx.x; item < a.n_seq * a.Hkv; item += gridDim.x) {
    const int s = a.by_Hkv.of(item), head = item - s * a.Hkv;
    int n = a.kv_lens[s];
    if (n < 0 || n > a.capacity || n > ((long long)a.table_pages << a.page_shift)) bad = true, n = 0;
    const float* w = a.weights + (long long)item * a.capacity;
    float* to = a.new_weights + (long long)item * a.budget;
    int32_t* kept = a.kept + (long long)item * a.budget;
    const int m = min(n, a.budget);
    if (head == 0 && threadIdx.x == 0) a.new_lens[s] = m;
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
    // --- the weight of the last key that is kept, and how many that have it are
    const int lo = a.first, hi = n - a.last;
    int need = a.budget - a.first - a.last; // of the keys lo .. hi - 1, fewer than there are
    uint32_t prefix = 0, mask = 0;
    if (need > 0) {
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 1024 : 2048;
        for (int i = threadIdx.x; i < kBins; i += kThreads) bins[i] = 0;
        __syncthreads();
        for (int i0 = lo; i0 < hi; i0 += kTile) {      // the loads of a tile before its counts
          uint32_t r[kEach];
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            const int i = i0 + j * kThreads + (int)threadIdx.x;
            r[j] = i < hi ? rank_of(w[i]) : 0u;
          }
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            const int i = i0 + j * kThreads + (int)threadIdx.x;
            if (i < hi && (r[j] & mask) == prefix) atomicAdd(&bins[(r[j] >> shift) & (width - 1)], 1);
          }
        }
        __syncthreads();
        // from the largest digit down: thread t has the digits below width - 4 t
        int own = 0, total;
#pragma unroll
        for (int j = 0; j < kBins / kThreads; ++j) {
          const int b = width - 1 - ((int)threadIdx.x * (kBins / kThreads) + j);
          own += b >= 0 ? bins[b] : 0;
        }
        int above = block_scan(own, warps, total);
        if (above < need && above + own >= need)
          for (int j = 0; j < kBins / kThreads; ++j) {
            const int b = width - 1 - ((int)threadIdx.x * (kBins / kThreads) + j);
            if (above + bins[b] >= need) {
              found[0] = b;
              found[1] = above;
              break;
            }
            above += bins[b];
          }
        __syncthreads();
        prefix |= (uint32_t)found[0] << shift;
        mask |= (uint32_t)(width - 1) << shift;
        need -= found[1];                   // of those that share the digits so far
        __syncthreads();
      }
    }
    // --- places, in key order; `need` keys of the weight `prefix` are kept, the first ones
    int at = 0, ties = 0;
    for (int i0 = 0; i0 < n; i0 += kTile) {
      float x[kEach];
      int gt[kEach], eq[kEach], eqs = 0, all;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int i = i0 + (int)threadIdx.x * kEach + j;
        x[j] = i < n ? w[i] : 0.f;
        const uint32_t r = rank_of(x[j]);
        const bool middle = i >= lo && i < hi;
        gt[j] = i < n && (!middle || (mask && r > prefix));
        eq[j] = middle && mask && r == prefix;
        eqs += eq[j];
      }
      int tie = ties + block_scan(eqs, warps, all);
      ties += all;
      int keep = 0;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        if (eq[j] && tie++ < need) gt[j] = 1;
        keep += gt[j];
      }
      int place = at + block_scan(keep, warps, all);
      at += all;
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        if (gt[j]) {
          to[place] = x[j];
          kept[place++] = i0 + (int)threadIdx.x * kEach + j;
        }
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) report(rep, blockIdx.x, any ? kStatusBounds : 0);
}

// Rows of the kept keys, 16 bytes of K and of V per thread
constexpr int kCopyThreads = 256;
template <int D>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictArgs a, const Report rep) {
  constexpr int kLanes = D / 8;
  pdl_wait();
  bool bad = false;
  const int lane = threadIdx.x % kLanes;
  const long long rows = (long long)a.n_seq * a.Hkv * a.budget;
  const int in_page = (1 << a.page_shift) - 1;
  for (long long r = ((long long)blockIdx.x * kCopyThreads + threadIdx.x) / kLanes; r < rows;
       r += (long long)gridDim.x * (kCopyThreads / kLanes)) {
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

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& a, void* ws, int num_sms, cudaStream_t stream) {
  const int items = a.n_seq * a.Hkv, grid = items < kFlagsFirst ? items : kFlagsFirst;
  const Report rep{ws, 0, {grid, 0}};
  evict_select_kernel<<<grid, kThreads, 0, stream>>>(a, rep);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const long long rows = (long long)items * a.budget, blocks = (rows * (a.D / 8) + kCopyThreads - 1) / kCopyThreads;
  const long long most = 16ll * num_sms;
  auto kern = a.D == 64 ? evict_copy_kernel<64> : evict_copy_kernel<128>;
  return launch_pdl(kern, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kCopyThreads), 0, stream, a, rep);
}

}  // namespace attn
}  // namespace moe
