// Device helpers and tensor maps shared by the attention kernels.
#pragma once

#include "attn.h"
#include "tc_ptx.cuh"

namespace moe {
namespace attn {
namespace {

using namespace tcx;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (kF16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes (the low or the high half of w) as f16
template <int kHalf>
__device__ __forceinline__ uint32_t codes2(uint32_t w) {
  uint32_t r;
  if (kHalf) asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}" : "=r"(r) : "r"(w));
  else asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(r) : "r"(w));
  return r;
}
// The bytes of a row of codes in a tile as TMA leaves it: 16-byte pieces
// swizzled by the row (128-byte rows by 128 bytes, 64-byte rows by 64)
template <int D>
__device__ __forceinline__ uint32_t code_at(uint32_t tile, int row, int byte) {
  const int piece = D == 128 ? (byte >> 4) ^ (row & 7) : (byte >> 4) ^ ((row >> 1) & 3);
  return tile + row * D + piece * 16 + (byte & 15);
}
__device__ __forceinline__ uint4 lds4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 half2_floats(uint32_t w) {
  float2 v;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(w));
  return v;
}
// Two bf16 elements
__device__ __forceinline__ float2 bf16_floats(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// Two fp32 values in one 64-bit register and the paired operations on them
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 64 columns of this lane's row; the values are there after tmem_wait_ld64
// on the same array (which ties the wait to them)
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&r)[64]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
               "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,"
               "%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,"
               "%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
                 "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]),
                 "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]),
                 "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]),
                 "=f"(r[29]), "=f"(r[30]), "=f"(r[31]), "=f"(r[32]), "=f"(r[33]), "=f"(r[34]), "=f"(r[35]),
                 "=f"(r[36]), "=f"(r[37]), "=f"(r[38]), "=f"(r[39]), "=f"(r[40]), "=f"(r[41]), "=f"(r[42]),
                 "=f"(r[43]), "=f"(r[44]), "=f"(r[45]), "=f"(r[46]), "=f"(r[47]), "=f"(r[48]), "=f"(r[49]),
                 "=f"(r[50]), "=f"(r[51]), "=f"(r[52]), "=f"(r[53]), "=f"(r[54]), "=f"(r[55]), "=f"(r[56]),
                 "=f"(r[57]), "=f"(r[58]), "=f"(r[59]), "=f"(r[60]), "=f"(r[61]), "=f"(r[62]), "=f"(r[63])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld64(float (&r)[64]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                 "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]),
                 "+f"(r[15]), "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]),
                 "+f"(r[22]), "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]),
                 "+f"(r[29]), "+f"(r[30]), "+f"(r[31]), "+f"(r[32]), "+f"(r[33]), "+f"(r[34]), "+f"(r[35]),
                 "+f"(r[36]), "+f"(r[37]), "+f"(r[38]), "+f"(r[39]), "+f"(r[40]), "+f"(r[41]), "+f"(r[42]),
                 "+f"(r[43]), "+f"(r[44]), "+f"(r[45]), "+f"(r[46]), "+f"(r[47]), "+f"(r[48]), "+f"(r[49]),
                 "+f"(r[50]), "+f"(r[51]), "+f"(r[52]), "+f"(r[53]), "+f"(r[54]), "+f"(r[55]), "+f"(r[56]),
                 "+f"(r[57]), "+f"(r[58]), "+f"(r[59]), "+f"(r[60]), "+f"(r[61]), "+f"(r[62]), "+f"(r[63])
               :
               : "memory");
}
// Every wait of the attention kernels gives up after this time (a poll may
// itself suspend the thread for a while, so polls are not counted).
constexpr uint64_t kWaitNs = 500000000;
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// A bounded wait that does not sleep between polls: for warps that the tensor
// cores or the softmax depend on.  One poll, then a rolled loop that reads the
// clock between polls: sixteen polls in a row were a quarter of the kernels'
// code (8192 causal 317 -> 306 us, 37 ragged prompts 27.9 -> 26.1, 16 sequences
// of D = 64 37.1 -> 34.9 when it was done).
__device__ __forceinline__ bool spin_wait(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = now_ns();
#pragma unroll 1
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (now_ns() - t0 > kWaitNs) return false;
  }
}
// The same for a converged warp: every lane polls, the verdict is uniform.
__device__ __forceinline__ bool warp_spin(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, spin_wait(bar, parity));
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
// One lane of a converged warp (the same one every time)
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e != 0;
}

// Keys [keys][D] as an operand of the product with queries: K-major, 128-byte swizzle,
// groups of 8 keys `group` bytes apart.
__device__ __forceinline__ uint64_t umma_desc_k(uint32_t saddr, uint32_t group) {
  return (umma_desc(saddr) & ~((uint64_t)0x3FFF << 32)) | (uint64_t)(group >> 4) << 32;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, int v,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(smem_u32(bar))
      : "memory");
}

// One box to global memory, as a bulk group of its own
__device__ __forceinline__ void store_box(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n"
      "cp.async.bulk.commit_group;" ::"l"(map),
      "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
      : "memory");
}

// ------------------------------------------------------------------ host side
inline bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box, CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  EncodeTiledFn fn = encode_fn();
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn && fn(m, type, rank, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D map over the queries: {D, head, token}; box {64, G, tt}.
inline bool q_map(CUtensorMap* m, const Heads& q, int T, int Hq, int Hkv, int D, int tt) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)T};
  const cuuint64_t strides[2] = {q.head * 2ull, q.tok * 2ull};
  const cuuint32_t box[3] = {64, (cuuint32_t)(Hq / Hkv), (cuuint32_t)tt};
  return encode(m, q.data, 3, dims, strides, box);
}

// Packed rows [tokens, heads, D] as {D, token, head}: a box of {64, rows, 1}
// is one 128-byte wide swizzled column of a tile.
inline bool rows_map(CUtensorMap* m, const Heads& v, const AttnArgs& a, long long tokens, int heads, int box) {
  const bool none = tokens == 0;       // nothing is ever loaded: any valid address
  const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)(none ? 1 : tokens), (cuuint64_t)(none ? 1 : heads)};
  const cuuint64_t strides[2] = {none ? a.D * 2ull : v.tok * 2ull, none ? a.D * 2ull : v.head * 2ull};
  const cuuint32_t boxd[3] = {64, (cuuint32_t)box, 1};
  return encode(m, none ? a.q.data : v.data, 3, dims, strides, boxd);
}

// A cache [pages, Hkv, page_size, D] as {64 of D, 8 rows, D / 64, rows / 8,
// page * Hkv + head}: one box of {64, 8, D / 64, rows / 8, 1} brings `rows`
// rows whole, as groups of 8 rows, each group D / 64 swizzled atoms of 1 KB.
// (With a box per 64 columns a 16-row page takes two boxes of 2 KB, and the
// copy engine spends ~95 cycles on a box: causal 8192 from 16-row pages then took
// 22% longer than from pages of 128; now 322 us against 316.)
inline bool pages_map(CUtensorMap* m, const uint16_t* cache, int D, int page_shift, int pages, int Hkv, int rows) {
  const cuuint64_t page = (cuuint64_t)D << page_shift;
  const cuuint64_t dims[5] = {64, 8, (cuuint64_t)D / 64, 1ull << (page_shift - 3), (cuuint64_t)pages * Hkv};
  const cuuint64_t strides[4] = {D * 2ull, 128, D * 16ull, page * 2};
  const cuuint32_t box[5] = {64, 8, (cuuint32_t)D / 64, (cuuint32_t)rows / 8, 1};
  return encode(m, cache, 5, dims, strides, box);
}
inline bool pages_map(CUtensorMap* m, const uint16_t* cache, const AttnArgs& a, int rows) {
  return pages_map(m, cache, a.D, a.page_shift, a.pages, a.Hkv, rows);
}

// A cache of codes [pages, Hkv, page_size, D] as {D, row, page * Hkv + head}: a
// box of {D, rows, 1} brings `rows` rows of D bytes, one after the other,
// swizzled by their own width.
inline bool codes_map(CUtensorMap* m, const void* cache, const AttnArgs& a, int rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)a.D, 1ull << a.page_shift, (cuuint64_t)a.pages * a.Hkv};
  const cuuint64_t strides[2] = {(cuuint64_t)a.D, (cuuint64_t)a.D << a.page_shift};
  const cuuint32_t box[3] = {(cuuint32_t)a.D, (cuuint32_t)rows, 1};
  return encode(m, cache, 3, dims, strides, box, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                a.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace
}  // namespace attn
}  // namespace moe
