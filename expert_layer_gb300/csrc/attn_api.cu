// C ABI of the attention operators: argument checks and launches.  Nothing
// here allocates, synchronises or keeps state between calls (but for the
// test-only setting of the waits).
#include <limits.h>
#include <stdint.h>

#include <atomic>

#include "moe.h"
#include "attn.h"
#include "common.cuh"

using namespace moe;
using namespace moe::attn;

namespace moe {
namespace attn {

int read_flags(const void* workspace) {
  Header h;
  if (cudaMemcpy(&h, workspace, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess) return -1;
  int bits = 0;
  for (int s = 0; s < kFlagSets; ++s) {
    if (h.blocks[s] < 0) return -1;
    const int* at = reinterpret_cast<const int*>(static_cast<const char*>(workspace) + sizeof(Header)) + s * kFlagsFirst;
    int words[1024];
    for (int done = 0; done < h.blocks[s];) {
      const int n = h.blocks[s] - done < 1024 ? h.blocks[s] - done : 1024;
      if (cudaMemcpy(words, at + done, sizeof(int) * n, cudaMemcpyDeviceToHost) != cudaSuccess) return -1;
      for (int i = 0; i < n; ++i) bits |= words[i];
      done += n;
    }
  }
  return bits;
}

}  // namespace attn
}  // namespace moe

namespace {

// Test-only (moe_debug_attn_wait_timeout)
std::atomic<int> g_hold{kHoldNone};

#define ATTN_TRY(expr)             \
  do {                             \
    const int _rc = (expr);        \
    if (_rc != MOE_OK) return _rc; \
  } while (0)

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int need16(const void* p) {
  if (!p) return MOE_ERR_INVALID_ARG;
  return aligned(p, 16) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}
int need4(const void* p) {
  if (!p) return MOE_ERR_INVALID_ARG;
  return aligned(p, 4) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

int check_shape(long long T, long long n_seq, long long Hq, long long Hkv, long long D) {
  if (T < 0 || n_seq < 0 || Hq <= 0 || Hkv <= 0 || D <= 0) return MOE_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return MOE_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return MOE_ERR_UNSUPPORTED;
  if (Hq / Hkv > 128 || Hq > 65536) return MOE_ERR_UNSUPPORTED;
  if (T * Hq >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_type(int dtype) { return dtype == MOE_BF16 || dtype == MOE_F16 ? MOE_OK : MOE_ERR_INVALID_ARG; }

// A [tokens, heads, D] view; the strides of a dimension of size one do not
// matter and are replaced by dense ones.
int check_heads(const moe_heads* v, long long tokens, int heads, int D, Heads* out) {
  if (!v) return MOE_ERR_INVALID_ARG;
  ATTN_TRY(need16(v->data));
  long long hs = v->head_stride, ts = v->token_stride;
  if (heads == 1) hs = D;
  if (tokens == 1) ts = (long long)heads * D;
  if (hs <= 0 || ts <= 0) return MOE_ERR_INVALID_ARG;
  if (hs % 8 != 0 || ts % 8 != 0 || hs >= (1ll << 38) || ts >= (1ll << 38)) return MOE_ERR_UNSUPPORTED;
  *out = Heads{static_cast<const uint16_t*>(v->data), ts, hs};
  return MOE_OK;
}

int check_cache(const moe_kv_cache* c, int* shift) {
  if (!c) return MOE_ERR_INVALID_ARG;
  ATTN_TRY(need16(c->k));
  ATTN_TRY(need16(c->v));
  if (c->pages <= 0 || c->page_size <= 0) return MOE_ERR_INVALID_ARG;
  int s = 4;
  while (s < 8 && (1 << s) != c->page_size) ++s;
  if ((1 << s) != c->page_size) return MOE_ERR_UNSUPPORTED;
  if ((long long)c->pages * c->page_size >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
  *shift = s;
  return MOE_OK;
}

int check_cache(const moe_kv_cache_fp8* c, int* shift) {
  if (!c) return MOE_ERR_INVALID_ARG;
  const moe_kv_cache plain{c->k, c->v, c->pages, c->page_size};
  ATTN_TRY(check_cache(&plain, shift));
  return need16(c->scales);
}

// What the two appends share: everything but where k and v go.  (Not for T = 0.)
int rope_args(RopeArgs& a, const moe_heads* q, const moe_heads* k, const moe_heads* v, const float* q_norm,
              const float* k_norm, float eps, const float* table, int max_pos, int rot, int interleaved,
              const int32_t* positions, const uint8_t* axes, int n_axes, int T, int Hq, int Hkv, int D, int dtype,
              void* q_out) {
  ATTN_TRY(check_heads(q, T, Hq, D, &a.q));
  ATTN_TRY(check_heads(k, T, Hkv, D, &a.k));
  ATTN_TRY(check_heads(v, T, Hkv, D, &a.v));
  if (rot > 0) ATTN_TRY(need16(table));
  if ((q_norm && !aligned(q_norm, 16)) || (k_norm && !aligned(k_norm, 16))) return MOE_ERR_UNSUPPORTED;
  ATTN_TRY(need4(positions));
  if (axes) ATTN_TRY(need4(axes));
  ATTN_TRY(need16(q_out));
  a.q_norm = q_norm; a.k_norm = k_norm; a.eps = eps;
  a.table = table; a.max_pos = max_pos; a.rot = rot; a.interleaved = interleaved != 0;
  a.positions = positions; a.axes = axes; a.n_axes = axes ? n_axes : 1;
  a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.f16 = dtype == MOE_F16;
  a.q_out = static_cast<uint16_t*>(q_out);
  return MOE_OK;
}

int check_rope(int rot, int D, int max_pos, float eps, const uint8_t* axes, int n_axes) {
  if (rot < 0 || rot > D || max_pos <= 0 || !(eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
  if (axes && n_axes < 1) return MOE_ERR_INVALID_ARG;
  if (rot % 16 != 0 || (axes && n_axes > kMaxAxes)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_device(int* num_sms) {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  return major == 10 && minor == 3 ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// One token per sequence: the shared prefix's parts on the tensor cores (the
// whole batch is one sequence of rows for it), then the rows' own keys.
int run_decode(const AttnArgs& a, const Layout& L, void* ws, int sms, cudaStream_t s) {
  DecodeParts p{};
  p.tc_o = ws_ptr<float>(ws, L.part_o);
  p.tc_lse = ws_ptr<float>(ws, L.part_lse);
  p.slot_o = ws_ptr<float>(ws, L.slot_o);
  p.slot_lse = ws_ptr<float>(ws, L.slot_lse);
  p.tail = ws_ptr<int4>(ws, L.tail);
  p.held = ws_ptr<int2>(ws, L.held);
  Report rep{ws, 0, {sms, 0}};
  int splits = 0;
  Beside beside{};
  if (a.prefix_len > 0) {
    splits = tc_splits(a, sms);
    rep.set = 1;
    rep.blocks[1] = tc_items(a, splits);
    ATTN_TRY(cuda_status(launch_attn_tc(a, splits, p.tc_o, p.tc_lse, rep, s)));
    beside.prefix = true;
    beside.few = rep.blocks[1] < sms ? sms - rep.blocks[1] : 0;
    beside.head = kHeadFixed + kHeadPerBlock * (((a.prefix_len + 127) / 128 + splits - 1) / splits);
    p.row_o = p.tc_o + (long long)splits * a.T * a.Hq * a.D;
    p.row_lse = p.tc_lse + (long long)splits * a.T * a.Hq;
  }
  rep.set = 0;
  ATTN_TRY(cuda_status(launch_attn_decode(a, beside, p, rep, sms, s)));
  return cuda_status(launch_attn_merge(a, splits, p, sms, s));
}

// The checks shared by the three attention calls, in the order of the others
// of the library: shape, empty batch, pointers, workspace, device.
int run_attn(AttnArgs& a, const moe_heads* q, int dtype, void* out, float* lse, void* workspace,
             size_t workspace_bytes, void* stream) {
  ATTN_TRY(check_heads(q, a.T, a.Hq, a.D, &a.q));
  ATTN_TRY(need16(out));
  if (lse && !aligned(lse, 4)) return MOE_ERR_UNSUPPORTED;
  ATTN_TRY(need16(workspace));
  if (!(a.scale == a.scale) || a.scale > 3.0e38f || a.scale < -3.0e38f) return MOE_ERR_INVALID_ARG;
  const Layout L = make_attn_layout(a.T, a.n_seq, a.Hq, a.Hkv, a.D);
  if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  int sms = 0;
  ATTN_TRY(check_device(&sms));
  a.f16 = dtype == MOE_F16;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.hold = g_hold.load(std::memory_order_relaxed);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (sms > kMaxBlocks) sms = kMaxBlocks;
  const Report rep{workspace, 1, {0, 0}};
  if (!a.q_starts) return run_decode(a, L, workspace, sms, s);
  const int splits = tc_splits(a, sms);
  if (splits == 1) return cuda_status(launch_attn_tc(a, 1, nullptr, nullptr, rep, s));
  DecodeParts p{};
  p.tc_o = ws_ptr<float>(workspace, L.part_o);
  p.tc_lse = ws_ptr<float>(workspace, L.part_lse);
  ATTN_TRY(cuda_status(launch_attn_tc(a, splits, p.tc_o, p.tc_lse, rep, s)));
  return cuda_status(launch_attn_merge(a, splits, p, 0, s));
}

const float* scales_of(const moe_kv_cache*) { return nullptr; }
const float* scales_of(const moe_kv_cache_fp8* c) { return c->scales; }

template <typename Cache>
int prefill_paged(const moe_heads* q, const Cache* cache, const int32_t* page_table, int table_pages,
                  const int32_t* q_starts, const int32_t* kv_lens, int n_seq, int T, int Hq, int Hkv, int D, int dtype,
                  int causal, float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                  void* stream) {
  ATTN_TRY(check_shape(T, n_seq, Hq, Hkv, D));
  ATTN_TRY(check_type(dtype));
  if (table_pages <= 0 || (T > 0 && n_seq == 0)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  AttnArgs a{};
  ATTN_TRY(check_cache(cache, &a.page_shift));
  ATTN_TRY(need4(page_table));
  ATTN_TRY(need4(q_starts));
  ATTN_TRY(need4(kv_lens));
  a.k_cache = static_cast<const uint16_t*>(cache->k);
  a.v_cache = static_cast<const uint16_t*>(cache->v);
  a.scales = scales_of(cache);
  if (a.scales && ((long long)table_pages << a.page_shift) > kMostIndex) return MOE_ERR_UNSUPPORTED;
  a.pages = cache->pages;
  a.page_table = page_table; a.table_pages = table_pages; a.q_starts = q_starts; a.kv_lens = kv_lens;
  a.n_seq = n_seq; a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.causal = causal != 0; a.scale = scale;
  return run_attn(a, q, dtype, out, lse, workspace, workspace_bytes, stream);
}

template <typename Cache>
int decode(const moe_heads* q, const Cache* cache, const int32_t* page_table, int table_pages, const int32_t* kv_lens,
           const int32_t* prefix_table, int prefix_len, int B, int Hq, int Hkv, int D, int dtype, float scale,
           void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  ATTN_TRY(check_shape(B, B, Hq, Hkv, D));
  ATTN_TRY(check_type(dtype));
  if (table_pages <= 0 || prefix_len < 0) return MOE_ERR_INVALID_ARG;
  if (B == 0) return MOE_OK;
  AttnArgs a{};
  ATTN_TRY(check_cache(cache, &a.page_shift));
  ATTN_TRY(need4(page_table));
  ATTN_TRY(need4(kv_lens));
  if (prefix_len > 0) ATTN_TRY(need4(prefix_table));
  if (prefix_len > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  a.k_cache = static_cast<const uint16_t*>(cache->k);
  a.v_cache = static_cast<const uint16_t*>(cache->v);
  a.scales = scales_of(cache);
  if (a.scales && ((long long)table_pages << a.page_shift) > kMostIndex) return MOE_ERR_UNSUPPORTED;
  a.pages = cache->pages;
  a.page_table = page_table; a.table_pages = table_pages; a.kv_lens = kv_lens;
  a.prefix_table = prefix_table; a.prefix_len = prefix_len;
  a.n_seq = B; a.T = B; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.scale = scale;
  if (!decode_fits(a)) return MOE_ERR_UNSUPPORTED;
  return run_attn(a, q, dtype, out, lse, workspace, workspace_bytes, stream);
}

}  // namespace

extern "C" {

size_t moe_attn_workspace_size(int T, int n_seq, int Hq, int Hkv, int D) {
  if (check_shape(T, n_seq, Hq, Hkv, D) != MOE_OK) return 0;
  return make_attn_layout(T, n_seq, Hq, Hkv, D).total;
}

int moe_debug_attn_wait_timeout(int wait) {
  if (wait < 0 || wait >= kHolds) return MOE_ERR_INVALID_ARG;
  g_hold.store(wait);
  return MOE_OK;
}

int moe_rope_append_axes(const moe_heads* q, const moe_heads* k, const moe_heads* v, const float* q_norm,
                         const float* k_norm, float eps, const float* table, int max_pos, int rot, int interleaved,
                         const int32_t* positions, const uint8_t* axes, int n_axes, const int32_t* slots, int T,
                         int Hq, int Hkv, int D, int dtype, void* q_out, const moe_kv_cache* cache, void* workspace,
                         size_t workspace_bytes, void* stream) {
  ATTN_TRY(check_shape(T, 0, Hq, Hkv, D));
  ATTN_TRY(check_type(dtype));
  ATTN_TRY(check_rope(rot, D, max_pos, eps, axes, n_axes));
  if (T == 0) return MOE_OK;
  RopeArgs a{};
  ATTN_TRY(rope_args(a, q, k, v, q_norm, k_norm, eps, table, max_pos, rot, interleaved, positions, axes, n_axes, T, Hq,
                     Hkv, D, dtype, q_out));
  ATTN_TRY(need4(slots));
  ATTN_TRY(check_cache(cache, &a.page_shift));
  ATTN_TRY(need16(workspace));
  if (workspace_bytes < make_attn_layout(T, 0, Hq, Hkv, D).total) return MOE_ERR_WORKSPACE;
  int sms = 0;
  ATTN_TRY(check_device(&sms));
  a.slots = slots;
  a.k_cache = static_cast<uint16_t*>(cache->k);
  a.v_cache = static_cast<uint16_t*>(cache->v);
  a.pages = cache->pages;
  return cuda_status(launch_rope_append(a, workspace, sms, static_cast<cudaStream_t>(stream)));
}

int moe_rope_append(const moe_heads* q, const moe_heads* k, const moe_heads* v, const float* q_norm,
                    const float* k_norm, float eps, const float* table, int max_pos, int rot, int interleaved,
                    const int32_t* positions, const int32_t* slots, int T, int Hq, int Hkv, int D, int dtype,
                    void* q_out, const moe_kv_cache* cache, void* workspace, size_t workspace_bytes,
                    void* stream) {
  return moe_rope_append_axes(q, k, v, q_norm, k_norm, eps, table, max_pos, rot, interleaved, positions, nullptr, 0,
                              slots, T, Hq, Hkv, D, dtype, q_out, cache, workspace, workspace_bytes, stream);
}

int moe_rope_append_fp8(const moe_heads* q, const moe_heads* k, const moe_heads* v, const float* q_norm,
                        const float* k_norm, float eps, const float* table, int max_pos, int rot, int interleaved,
                        const int32_t* positions, const uint8_t* axes, int n_axes, const int32_t* page_table,
                        int table_pages, const int32_t* q_starts, const int32_t* kv_lens, int n_seq, int T, int Hq,
                        int Hkv, int D, int dtype, void* q_out, const moe_kv_cache_fp8* cache, void* workspace,
                        size_t workspace_bytes, void* stream) {
  ATTN_TRY(check_shape(T, n_seq, Hq, Hkv, D));
  ATTN_TRY(check_type(dtype));
  ATTN_TRY(check_rope(rot, D, max_pos, eps, axes, n_axes));
  if (table_pages <= 0 || (T > 0 && n_seq == 0)) return MOE_ERR_INVALID_ARG;
  if (n_seq >= (1 << 28)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  RopeFp8Args f{};
  ATTN_TRY(rope_args(f.r, q, k, v, q_norm, k_norm, eps, table, max_pos, rot, interleaved, positions, axes, n_axes, T,
                     Hq, Hkv, D, dtype, q_out));
  ATTN_TRY(check_cache(cache, &f.r.page_shift));
  ATTN_TRY(need4(page_table));
  ATTN_TRY(need4(q_starts));
  ATTN_TRY(need4(kv_lens));
  ATTN_TRY(need16(workspace));
  if (workspace_bytes < make_attn_layout(T, n_seq, Hq, Hkv, D).total) return MOE_ERR_WORKSPACE;
  int sms = 0;
  ATTN_TRY(check_device(&sms));
  f.k_codes = static_cast<uint8_t*>(cache->k);
  f.v_codes = static_cast<uint8_t*>(cache->v);
  f.scales = cache->scales;
  f.r.pages = cache->pages;
  f.page_table = page_table; f.table_pages = table_pages; f.q_starts = q_starts; f.kv_lens = kv_lens;
  f.n_seq = n_seq;
  return cuda_status(launch_rope_append_fp8(f, workspace, sms, static_cast<cudaStream_t>(stream)));
}

int moe_attn_prefill(const moe_heads* q, const moe_heads* k, const moe_heads* v, const int32_t* q_starts,
                     const int32_t* kv_starts, int n_seq, int T, int Tk, int Hq, int Hkv, int D, int dtype,
                     int causal, float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                     void* stream) {
  ATTN_TRY(check_shape(T, n_seq, Hq, Hkv, D));
  ATTN_TRY(check_type(dtype));
  if (Tk < 0 || (T > 0 && n_seq == 0)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  AttnArgs a{};
  if (Tk > 0) {   // without any key every row is empty and k and v are not read
    ATTN_TRY(check_heads(k, Tk, Hkv, D, &a.k));
    ATTN_TRY(check_heads(v, Tk, Hkv, D, &a.v));
  }
  ATTN_TRY(need4(q_starts));
  ATTN_TRY(need4(kv_starts));
  a.q_starts = q_starts; a.kv_starts = kv_starts;
  a.n_seq = n_seq; a.T = T; a.Tk = Tk; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.causal = causal != 0; a.scale = scale;
  return run_attn(a, q, dtype, out, lse, workspace, workspace_bytes, stream);
}

int moe_attn_prefill_paged(const moe_heads* q, const moe_kv_cache* cache, const int32_t* page_table,
                           int table_pages, const int32_t* q_starts, const int32_t* kv_lens, int n_seq, int T,
                           int Hq, int Hkv, int D, int dtype, int causal, float scale, void* out, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream) {
  return prefill_paged(q, cache, page_table, table_pages, q_starts, kv_lens, n_seq, T, Hq, Hkv, D, dtype, causal, scale,
                       out, lse, workspace, workspace_bytes, stream);
}

int moe_attn_prefill_paged_fp8(const moe_heads* q, const moe_kv_cache_fp8* cache, const int32_t* page_table,
                               int table_pages, const int32_t* q_starts, const int32_t* kv_lens, int n_seq, int T,
                               int Hq, int Hkv, int D, int dtype, int causal, float scale, void* out, float* lse,
                               void* workspace, size_t workspace_bytes, void* stream) {
  return prefill_paged(q, cache, page_table, table_pages, q_starts, kv_lens, n_seq, T, Hq, Hkv, D, dtype, causal, scale,
                       out, lse, workspace, workspace_bytes, stream);
}

int moe_attn_decode(const moe_heads* q, const moe_kv_cache* cache, const int32_t* page_table, int table_pages,
                    const int32_t* kv_lens, const int32_t* prefix_table, int prefix_len, int B, int Hq, int Hkv,
                    int D, int dtype, float scale, void* out, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream) {
  return decode(q, cache, page_table, table_pages, kv_lens, prefix_table, prefix_len, B, Hq, Hkv, D, dtype, scale, out,
                lse, workspace, workspace_bytes, stream);
}

int moe_attn_decode_fp8(const moe_heads* q, const moe_kv_cache_fp8* cache, const int32_t* page_table, int table_pages,
                        const int32_t* kv_lens, const int32_t* prefix_table, int prefix_len, int B, int Hq, int Hkv,
                        int D, int dtype, float scale, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, void* stream) {
  return decode(q, cache, page_table, table_pages, kv_lens, prefix_table, prefix_len, B, Hq, Hkv, D, dtype, scale, out,
                lse, workspace, workspace_bytes, stream);
}

int moe_attn_key_weights(const moe_heads* q, const void* k_cache, int pages, int page_size, const int32_t* page_table,
                         int table_pages, const int32_t* q_starts, const int32_t* kv_lens, int n_seq, int T, int Hq,
                         int Hkv, int D, int dtype, int causal, float scale, const float* lse, float* weights,
                         int capacity, void* workspace, size_t workspace_bytes, void* stream) {
  ATTN_TRY(check_shape(T, n_seq, Hq, Hkv, D));
  ATTN_TRY(check_type(dtype));
  if (table_pages <= 0 || capacity <= 0 || (T > 0 && n_seq == 0)) return MOE_ERR_INVALID_ARG;
  if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f) return MOE_ERR_INVALID_ARG;
  if (capacity > kMostIndex || (long long)n_seq * Hkv > kMostIndex) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  WeightArgs a{};
  ATTN_TRY(check_heads(q, T, Hq, D, &a.q));
  const moe_kv_cache keys{const_cast<void*>(k_cache), const_cast<void*>(k_cache), pages, page_size};
  ATTN_TRY(check_cache(&keys, &a.page_shift));
  ATTN_TRY(need4(page_table));
  ATTN_TRY(need4(q_starts));
  ATTN_TRY(need4(kv_lens));
  ATTN_TRY(need4(lse));
  ATTN_TRY(need4(weights));
  ATTN_TRY(need16(workspace));
  if (workspace_bytes < make_attn_layout(T, n_seq, Hq, Hkv, D).total) return MOE_ERR_WORKSPACE;
  int sms = 0;
  ATTN_TRY(check_device(&sms));
  if (sms > kMaxBlocks) sms = kMaxBlocks;
  a.k_cache = static_cast<const uint16_t*>(k_cache);
  a.page_table = page_table; a.q_starts = q_starts; a.kv_lens = kv_lens;
  a.table_pages = table_pages; a.pages = pages;
  a.n_seq = n_seq; a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.f16 = dtype == MOE_F16; a.causal = causal != 0;
  a.c = scale * 1.4426950408889634f;
  a.lse = lse; a.weights = weights; a.capacity = capacity;
  a.by_G.set(Hq / Hkv);
  a.hold = g_hold.load(std::memory_order_relaxed);
  return cuda_status(launch_attn_weights(a, workspace, sms, static_cast<cudaStream_t>(stream)));
}

int moe_kv_evict(const moe_kv_cache* cache, const int32_t* page_table, int table_pages, const int32_t* kv_lens,
                 const float* weights, int capacity, const int32_t* out_table, int out_pages, int budget,
                 int keep_first, int keep_last, int n_seq, int Hkv, int D, int32_t* new_lens, float* new_weights,
                 int32_t* kept, void* workspace, size_t workspace_bytes, void* stream) {
  ATTN_TRY(check_shape(0, n_seq, Hkv, Hkv, D));
  if (table_pages <= 0 || capacity <= 0 || out_pages <= 0 || budget <= 0 || keep_first < 0 || keep_last < 0)
    return MOE_ERR_INVALID_ARG;
  if ((long long)keep_first + keep_last > budget) return MOE_ERR_INVALID_ARG;
  if (capacity > kMostIndex || budget > kMostIndex || (long long)n_seq * Hkv > kMostIndex) return MOE_ERR_UNSUPPORTED;
  if (n_seq == 0) return MOE_OK;
  EvictArgs a{};
  ATTN_TRY(check_cache(cache, &a.page_shift));
  if (budget > ((long long)out_pages << a.page_shift)) return MOE_ERR_INVALID_ARG;
  ATTN_TRY(need4(page_table));
  ATTN_TRY(need4(out_table));
  ATTN_TRY(need4(kv_lens));
  ATTN_TRY(need4(weights));
  ATTN_TRY(need4(new_lens));
  ATTN_TRY(need4(new_weights));
  ATTN_TRY(need4(kept));
  ATTN_TRY(need16(workspace));
  if (workspace_bytes < make_attn_layout(0, n_seq, Hkv, Hkv, D).total) return MOE_ERR_WORKSPACE;
  int sms = 0;
  ATTN_TRY(check_device(&sms));
  a.k_cache = static_cast<uint16_t*>(cache->k);
  a.v_cache = static_cast<uint16_t*>(cache->v);
  a.page_table = page_table; a.out_table = out_table; a.kv_lens = kv_lens; a.weights = weights;
  a.table_pages = table_pages; a.out_pages = out_pages; a.pages = cache->pages; a.capacity = capacity;
  a.n_seq = n_seq; a.Hkv = Hkv; a.D = D;
  a.budget = budget; a.first = keep_first; a.last = keep_last;
  a.new_lens = new_lens; a.new_weights = new_weights; a.kept = kept;
  a.by_Hkv.set(Hkv);
  a.by_budget.set(budget);
  return cuda_status(launch_kv_evict(a, workspace, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
