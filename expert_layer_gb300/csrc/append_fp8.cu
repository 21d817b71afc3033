// Query / key norms, rotary positions and the append to a paged cache in 8
// bits: rope_append.cu's rows, with k and v as e4m3 codes and a scale 2^e for
// each 16 tokens of a page and head (attn.h).
//
// For the new rows of a scale block, k rotated or v, fp32:
//   need = smallest e with max |x| <= 448 * 2^e, from kScaleMin to kScaleMax
//   e    = max(need, the block's e) when rows of before are in it, else need
//   code = e4m3(x 2^-e), nearest even, at most 448; NaN stays NaN
// and, where e grew, the codes of before times 2^(old - e), rounded again (exact
// unless they become subnormal, below 2^-6 of the new scale).  Rows behind the
// sequence's end stay as they were.
//
// Bound: HBM for many tokens, latency for few, as rope_append.cu.  The rows of a
// scale block need one maximum, so one warp takes a (block, head, k or v): its 16
// rows wait in shared memory as they were loaded, turned once for the maximum
// and once more for the codes (the arithmetic is cheap; 16 rows in fp32
// registers spilled).  What a block holds follows from the lengths, so the call takes
// page tables and lengths instead of a slot for each token: no atomics, no
// second pass over the batch, the same bits every time.
// Measured (32 + 2 x 4 heads of 128, norms): 256 sequences with a token each 5.2
// us, 8 prompts of 700 to 1300 tokens 39.3 us = 4.2 TB/s, with DRAM 39% and the issue
// slots 50% busy: the loads' latency, mostly.  Not kept: two warps to a scale block,
// with its rows in registers, 41.7 us (64 registers) and 44.9 (80), from shared memory
// 40.8 and 43.2; the blocks of k and v between those of q 38.5 to 40.4.  (64 registers
// are a few short here too: 36 to 52 bytes spilled.)
#include "attn.h"
#include "attn_ptx.cuh"
#include "rope_rows.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = kRopeThreads;
constexpr int kWarps = kThreads / 32;
constexpr int kMany = 4;            // q heads per group of lanes once there are enough of them
constexpr int kResident = 4;

// The smallest e with top <= 448 * 2^e (448 = 1.75 * 2^8), within the range
__device__ __forceinline__ int needed_exp(float top) {
  const uint32_t b = __float_as_uint(top);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < kScaleMin ? kScaleMin : e > kScaleMax ? kScaleMax : e;
}

// Four values to e4m3 (finite ones beyond 448 become 448)
__device__ __forceinline__ uint32_t to_codes(uint64_t a, uint64_t b) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
      " mov.b32 %0, {l, h};\n}"
      : "=r"(r)
      : "f"(lo(a)), "f"(hi(a)), "f"(lo(b)), "f"(hi(b)));
  return r;
}
// Four codes times f (a power of two), rounded again
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float f) {
  uint32_t p, q;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(p), "=r"(q)
      : "r"(w));
  const uint64_t f2 = pair(f, f);
  return to_codes(mul2(unpack2<true>(p), f2), mul2(unpack2<true>(q), f2));
}

// Eight bytes to shared memory, or zeros
__device__ __forceinline__ void load8(void* dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 8 : 0)
               : "memory");
}

// Slots of the scale blocks that the sequences touch, enough of them without a
// prefix sum over the batch: n tokens touch at most n blocks, and at most
// n / 16 + 2.
__device__ __forceinline__ int slot_base(const RopeFp8Args& f, int s) {
  const int q = max(0, f.q_starts[s]);
  return f.by_token ? q : q / kScaleBlock + 2 * s;
}
// The last sequence whose slots begin at or before `slot`: all lanes of the warp search together.
__device__ __forceinline__ int slot_seq(const RopeFp8Args& f, int slot) {
  const int lane = threadIdx.x & 31;
  // (a batch of single tokens: sequence s has slot s)
  if (f.by_token && f.n_seq == f.r.T && slot < f.n_seq && f.q_starts[slot] == slot && f.q_starts[slot + 1] == slot + 1)
    return slot;
  int first = 0, n = f.n_seq;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool at = lane * step < n && slot_base(f, first + lane * step) <= slot;
    const int hit = 31 - __clz((int)(__ballot_sync(0xffffffffu, at) | 1u));
    first += hit * step;
    n = min(step, n - hit * step);
  }
  return first;
}

// The scale blocks of block `block` of `blocks`, a warp per (scale block, head, k or v).
template <int D, bool kF16, bool kInter>
__device__ __forceinline__ bool append_blocks(const RopeFp8Args& f, const bool axes, unsigned block, unsigned blocks) {
  constexpr int kLanes = D / (2 * kPart), kRows = 32 / kLanes, kPasses = kScaleBlock / kRows;
  __shared__ uint2 rows_of[kWarps][kPasses][2][32];      // [..][part][lane]: read by the lane that loaded it
  const RopeArgs& a = f.r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const LanePlace<kInter> at(a, lane % kLanes);
  const int sub = lane / kLanes;                       // row of a pass
  uint32_t which;
  bool bad = !lane_axes(a, axes, at, which);
  const long long room = (long long)f.table_pages << a.page_shift;
  if (block == 0) {
    if (threadIdx.x == 0) bad |= f.q_starts[0] != 0 || f.q_starts[f.n_seq] != a.T;
    for (int s = threadIdx.x; s < f.n_seq; s += kThreads) {
      const int q0 = f.q_starts[s], q1 = f.q_starts[s + 1], n = f.kv_lens[s];
      bad |= q0 < 0 || q1 < q0 || q1 > a.T || n < q1 - q0 || n > room;
    }
  }
  const int slots = f.by_token ? a.T : a.T / kScaleBlock + 2 * f.n_seq;
  const long long items = 2ll * slots * a.Hkv, warps = (long long)blocks * kWarps;
  const long long each = (items + warps - 1) / warps;
  const long long i0 = ((long long)block * kWarps + warp) * each, i1 = min(items, i0 + each);
  int seen = -1, q0 = 0, len = 0, fresh = 0, first = -1;             // of the slot in use
  const int32_t* list = nullptr;
#pragma unroll 1
  for (long long i = i0; i < i1; ++i) {
    const int slot = i >> 31 ? (int)(i / (2 * a.Hkv)) : f.by_Hkv2.of((int)i);
    const int part = (int)(i - (long long)slot * 2 * a.Hkv), head = part >> 1;
    const bool value = part & 1;
    if (slot != seen) {
      seen = slot;
      const int s = slot_seq(f, slot);
      q0 = f.q_starts[s];
      const int q1 = f.q_starts[s + 1];
      len = f.kv_lens[s];
      list = f.page_table + (long long)s * f.table_pages;
      first = -1;
      if (q0 >= 0 && q1 > q0 && q1 <= a.T && len >= q1 - q0 && len <= room) {
        fresh = len - (q1 - q0);                       // the first new token
        const long long b = (long long)(fresh / kScaleBlock) + slot - slot_base(f, s);
        if (b >= 0 && b * kScaleBlock < len) first = (int)b * kScaleBlock;   // (else a slot that the sequence does not need)
      }
    }
    if (first < 0) continue;
    const int r0 = max(0, fresh - first), r1 = min(kScaleBlock, len - first);      // the new rows
    const int p0 = r0 / kRows, p1 = (r1 + kRows - 1) / kRows;
    // --- the rows as they were loaded
    const Heads& src = value ? a.v : a.k;
    const uint16_t* in = src.data + head * src.head;
#pragma unroll 1
    for (int p = p0; p < p1; ++p) {                      // rows that are not there are zeros
      const int r = p * kRows + sub;
      const bool there = r >= r0 && r < r1;
      const uint16_t* row = in + (there ? (long long)(q0 + first + r - fresh) * src.tok : 0);
      load8(&rows_of[warp][p][0][lane], row + at.o1, there);
      load8(&rows_of[warp][p][1][lane], row + at.o2, there);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    const int page = list[first >> a.page_shift];
    // positions: lane r has those of row r
    Places mine;
    bool placed = true;
    {
#pragma unroll
      for (int x = 0; x < kMaxAxes; ++x) mine.p[x] = 0;
      if (lane >= r0 && lane < r1) placed = mine.load(a, axes, q0 + first + lane - fresh);
      if (!placed) {
        bad = true;
#pragma unroll
        for (int x = 0; x < kMaxAxes; ++x) mine.p[x] = 0;
      }
    }
    const uint32_t lost = __ballot_sync(0xffffffffu, !placed);     // rows that are not written
    if ((unsigned)page >= (unsigned)a.pages) {
      bad = true;
      asm volatile("cp.async.wait_all;" ::: "memory");
      continue;
    }
    const long long at_row = (((long long)page * a.Hkv + head) << a.page_shift) + (first & ((1 << a.page_shift) - 1));
    uint8_t* codes = (value ? f.v_codes : f.k_codes) + at_row * D;
    float* scale = f.scales + (at_row / kScaleBlock) * 2 + (value ? 1 : 0);
    const int old = r0 > 0 ? scale_exp(*scale) : kScaleMin;        // rows of before
    auto row_values = [&](int p, uint64_t (&y)[kPart]) {
      Part raw[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint2 v = rows_of[warp][p][x][lane];
        raw[x].w[0] = v.x, raw[x].w[1] = v.y;
      }
      if (value) {
#pragma unroll
        for (int j = 0; j < kPart; ++j) y[j] = unpack2<kF16>(raw[j / (kPart / 2)].w[j % (kPart / 2)]);
        return;
      }
      Places pos;
#pragma unroll
      for (int x = 0; x < kMaxAxes; ++x) pos.p[x] = __shfl_sync(0xffffffffu, mine.p[x], p * kRows + sub);
      float c[2 * kPart], s[2 * kPart];
      coefficients(a, axes, at, which, pos, a.k_norm, c, s);
      turn<D, kF16, kInter>(raw, a.k_norm != nullptr, a.k_norm != nullptr, a.eps, at.turns, c, s, y);
    };
    asm volatile("cp.async.wait_all;" ::: "memory");
    float top = 0.f;
#pragma unroll 2
    for (int p = p0; p < p1; ++p) {
      uint64_t y[kPart];
      row_values(p, y);
      if ((lost >> (p * kRows + sub)) & 1) continue;
#pragma unroll
      for (int j = 0; j < kPart; ++j) top = fmaxf(top, fmaxf(fabsf(lo(y[j])), fabsf(hi(y[j]))));   // NaN is passed over
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const int e = max(needed_exp(top), old);
    const uint64_t to = pair(exp2i(-e), exp2i(-e));
#pragma unroll 2
    for (int p = p0; p < p1; ++p) {
      uint64_t y[kPart];
      row_values(p, y);
      const int r = p * kRows + sub;
      if (r < r0 || r >= r1 || ((lost >> r) & 1)) continue;
      uint8_t* dst = codes + r * D;
      *reinterpret_cast<uint32_t*>(dst + at.o1) = to_codes(mul2(y[0], to), mul2(y[1], to));
      *reinterpret_cast<uint32_t*>(dst + at.o2) = to_codes(mul2(y[2], to), mul2(y[3], to));
    }
    if (e > old) {
      const float g = exp2i(old - e);
      for (int r = sub; r < r0; r += kRows) {
        uint2* w = reinterpret_cast<uint2*>(codes + r * D + (lane % kLanes) * 8);
        const uint2 v = *w;
        *w = make_uint2(rescaled(v.x, g), rescaled(v.y, g));
      }
    }
    if (lane == 0) *scale = exp2i(e);
  }
  return bad;
}

template <int D, int kHeads, bool kF16, bool kInter>
__global__ void __launch_bounds__(kThreads, kResident)
    append_fp8_kernel(const RopeFp8Args f, const Report rep) {
  const bool axes = f.r.axes != nullptr;
  const bool bad = (int)blockIdx.x < f.kv_blocks
                       ? append_blocks<D, kF16, kInter>(f, axes, blockIdx.x, f.kv_blocks)
                       : rope_rows<D, kHeads, kF16, kInter, false>(f.r, axes, blockIdx.x - f.kv_blocks,
                                                                   gridDim.x - f.kv_blocks);
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) report(rep, blockIdx.x, any ? kStatusBounds : 0);
}

template <int D, int kHeads, bool kF16>
cudaError_t launch(RopeFp8Args f, void* ws, int num_sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  RopeArgs& a = f.r;
  a.chunks = (a.Hq + kHeads - 1) / kHeads;
  a.by_chunks.set(a.chunks);
  const long long by16 = a.T / kScaleBlock + 2ll * f.n_seq;
  f.by_token = a.T <= by16;
  f.by_Hkv2.set(2 * a.Hkv);
  const long long q = ((long long)a.T * a.chunks + kGroups - 1) / kGroups;
  const long long kv = ((f.by_token ? a.T : by16) * 2 * a.Hkv + kWarps - 1) / kWarps;
  // k and v first, a warp for each scale block as far as the report's words go:
  // a block of them is a chain of loads, which the rows of q then cover (with
  // shares of one round of blocks by what is read, three or more scale blocks
  // to a warp, 256 tokens took 19.0 us, 8 prompts of 1000 56.6)
  const long long most = (long long)num_sms * kResident;
  const long long nq = q < most ? q : most < kFlagsFirst / 2 ? most : kFlagsFirst / 2;
  const long long nkv = kv < kFlagsFirst - nq ? kv : kFlagsFirst - nq;
  f.kv_blocks = (int)nkv;
  const int grid = (int)(nq + nkv);
  const Report rep{ws, 0, {grid, 0}};
  auto kern = a.interleaved ? append_fp8_kernel<D, kHeads, kF16, true> : append_fp8_kernel<D, kHeads, kF16, false>;
  kern<<<grid, kThreads, 0, stream>>>(f, rep);
  return cudaGetLastError();
}

template <int D, int kHeads>
cudaError_t launch_type(const RopeFp8Args& f, void* ws, int num_sms, cudaStream_t stream) {
  return f.r.f16 ? launch<D, kHeads, true>(f, ws, num_sms, stream) : launch<D, kHeads, false>(f, ws, num_sms, stream);
}

}  // namespace

cudaError_t launch_rope_append_fp8(const RopeFp8Args& f, void* ws, int num_sms, cudaStream_t stream) {
  const RopeArgs& a = f.r;
  // several heads to a group once that still gives every SM 512 threads (rope_append.cu)
  const bool many = (long long)a.T * a.Hq * (a.D / 8) / kMany >= 512ll * num_sms;
  if (a.D == 64)
    return many ? launch_type<64, kMany>(f, ws, num_sms, stream) : launch_type<64, 1>(f, ws, num_sms, stream);
  return many ? launch_type<128, kMany>(f, ws, num_sms, stream) : launch_type<128, 1>(f, ws, num_sms, stream);
}

}  // namespace attn
}  // namespace moe
