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
// A wait that does not sleep between polls (bounded as mbar_wait): for warps
// that the tensor cores or the softmax depend on.
__device__ __forceinline__ bool spin_wait(uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < kSpinLimit; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}

// The same for a converged warp: every lane polls, the verdict is uniform.
__device__ __forceinline__ bool warp_spin(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, spin_wait(bar, parity));
}
// One lane of a converged warp (the same one every time)
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e != 0;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// ------------------------------------------------------------------ host side
// 4-D map over keys or values: {D, row, head, page}; box {64, rows, 1, 1}.
inline bool kv_map(CUtensorMap* m, const AttnArgs& a, const uint16_t* cache, const Heads& packed, int box) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4], strides[3];
  const void* base;
  if (a.page_table) {
    const cuuint64_t page = (cuuint64_t)a.D << a.page_shift;
    dims[0] = a.D; dims[1] = 1ull << a.page_shift; dims[2] = a.Hkv; dims[3] = a.pages;
    strides[0] = a.D * 2ull; strides[1] = page * 2; strides[2] = page * 2 * a.Hkv;
    base = cache;
  } else {
    dims[0] = a.D; dims[1] = a.Tk > 0 ? a.Tk : 1; dims[2] = a.Hkv; dims[3] = 1;
    const bool none = a.Tk == 0;       // no key is ever loaded: any valid address
    strides[0] = none ? a.D * 2ull : packed.tok * 2ull;
    strides[1] = none ? a.D * 2ull : packed.head * 2ull;
    strides[2] = strides[0];
    base = none ? a.q.data : packed.data;
    if (none) dims[2] = 1;
  }
  const cuuint32_t boxd[4] = {64, (cuuint32_t)box, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, boxd, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace attn
}  // namespace moe
