// Attention operators: argument structs of the kernels, the workspace of an
// attention call and the host-side launchers.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"

namespace moe {
namespace attn {

// ------------------------------------------------------------- workspace
// Header of an attention call's workspace.  Its kernels report what they
// found in one word per block, written by every block: nothing has to be
// cleared before a call, so a call is not preceded by a clearing kernel.
// `magic` sits where the layer calls keep their status word and holds a value
// that no set of kStatus* bits can have.
constexpr int kHeaderMagic = 0x41540000;
constexpr int kFlagSets = 2;           // kernels of one call that report
constexpr int kFlagsFirst = 2048;      // blocks of set 0; those of set 1 follow, as many as a shape can have
struct Header {
  int magic;
  int blocks[kFlagSets];               // words in use of each set
  int pad[61];
};
static_assert(sizeof(Header) == sizeof(WsHeader), "header is one 256-byte slot");

// Rows of the partial results of calls whose key axis is split over blocks:
// at most two tiles of 128 rows per block of a grid (attn_tc.cu), or one per
// row and block where a call has fewer.  kMaxBlocks bounds the SMs of a GPU.
constexpr long long kMaxBlocks = 160;
constexpr long long kTileRows = 256;

struct Layout {
  size_t hdr, flags, part_o, part_lse, slot_o, slot_lse, tail, held, total;
};

inline Layout make_attn_layout(long long T, long long n_seq, long long Hq, long long Hkv, long long D) {
  Layout L{};
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t r = o; o = align256(o + bytes); return r; };
  const long long single = (T < n_seq ? T : n_seq) * Hq;    // rows of a decode batch
  long long rows = (T * Hq < kTileRows ? T * Hq : kTileRows) * kMaxBlocks;
  if (rows < single) rows = single;
  rows += single;                            // decode: one part more for each row's own keys
  L.hdr = take(sizeof(Header));
  const long long per = 2 * (128 / (Hq / Hkv));               // tokens of an attn_tc.cu block
  const long long items = (T / per + n_seq + 1) * Hkv;
  L.flags = take(sizeof(int) * (kFlagsFirst + (items > kMaxBlocks ? items : kMaxBlocks)));
  L.part_o = take(sizeof(float) * (size_t)rows * D);
  L.part_lse = take(sizeof(float) * (size_t)rows);
  L.slot_o = take(sizeof(float) * 2 * kMaxBlocks * 16 * D);
  L.slot_lse = take(sizeof(float) * 2 * kMaxBlocks * 16);
  L.tail = take(sizeof(int4) * kMaxBlocks);
  L.held = take(sizeof(int2) * (size_t)n_seq * Hkv * ((Hq / Hkv + 15) / 16));
  L.total = o;
  return L;
}

// OR of the words that the kernels of the last call left (the stream is idle);
// -1 when the copy fails
int read_flags(const void* workspace);

// Where a kernel of a call reports: its own set of words
struct Report {
  void* ws;
  int set;
  int blocks[kFlagSets];
};

// Every block of a reporting kernel does this (one thread), whatever it found:
// the words of a call are complete when its kernels are.
__device__ __forceinline__ void report(const Report& r, int block, int bits) {
  int* flags = reinterpret_cast<int*>(reinterpret_cast<char*>(r.ws) + sizeof(Header));
  flags[r.set * kFlagsFirst + block] = bits;
  if (block == 0) {
    Header* h = reinterpret_cast<Header*>(r.ws);
    h->magic = kHeaderMagic;
    for (int i = 0; i < kFlagSets; ++i) h->blocks[i] = r.blocks[i];
  }
}

// ------------------------------------------------------------- arguments
struct Heads {                // [tokens, heads, D], strides in elements
  const uint16_t* data;
  long long tok, head;
};

// Quotients of n in [0, 2^31) by a divisor that the host knows: with
// 2^(k-1) < d <= 2^k, m = ceil(2^(31+k) / d) < 2^32, n / d = floor(m n / 2^(31+k)):
// the error of m, less than one part in 2^31 of a quotient's unit, moves no
// quotient.  (A division is some 20 instructions, and those of a first item
// come from L2 as they run.)
struct Divisor {
  uint32_t m, shift;      // m = 0: d = 1
  void set(uint32_t d) {
    shift = 0;
    while ((1ull << (shift + 1)) < d) ++shift;
    m = d == 1 ? 0 : (uint32_t)(((1ull << (32 + shift)) + d - 1) / d);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int of(int n) const { return m ? (int)(__umulhi((uint32_t)n, m) >> shift) : n; }
#endif
};

constexpr int kMaxAxes = 4;

// Keys of a sequence, heads of a batch: their 32-bit indices are rounded up to a
// tile and stepped by a block's tile or a grid's blocks, 2^14 at most
constexpr long long kMostIndex = (1ll << 31) - (1 << 16);

struct RopeArgs {
  Heads q, k, v;
  const float* q_norm;        // [D] or null
  const float* k_norm;
  float eps;
  const float* table;         // [max_pos, rot]: cos | sin
  int max_pos, rot, interleaved;
  const uint8_t* axes;        // [rot / 2]: the row of `positions` that turns each pair; null: one row
  int n_axes;                 // at most kMaxAxes
  const int32_t* positions;   // [n_axes, T]
  const int32_t* slots;
  int T, Hq, Hkv, D, f16;
  uint16_t* q_out;            // [T, Hq, D]
  uint16_t* k_cache;          // [pages, Hkv, page_size, D]
  uint16_t* v_cache;
  int pages, page_shift;      // page_size = 1 << page_shift
  unsigned chunks;            // groups of heads of a token (the kernel's)
  Divisor by_chunks;
};

// ------------------------------------------------------------- the cache in 8 bits
// e4m3 codes and one scale 2^e per kScaleBlock tokens of a page and key-value
// head, of the keys and of the values: scales [pages, Hkv, page_size / 16, 2].
// A power of two costs a floating code nothing, and leaves every product with
// it, and every change of it, exact (but for codes that become subnormal).
// 57344 = 448 * 2^7 is the largest value, below f16's; 2^-24 * 2^-9 the
// smallest step.
constexpr int kScaleBlock = 16;
constexpr int kScaleMin = -24, kScaleMax = 7;

struct RopeFp8Args {
  RopeArgs r;                 // without slots and cache
  uint8_t* k_codes;           // [pages, Hkv, page_size, D]
  uint8_t* v_codes;
  float* scales;
  const int32_t* page_table;  // [n_seq, table_pages]
  const int32_t* q_starts;    // [n_seq + 1]
  const int32_t* kv_lens;     // [n_seq], with the call's tokens
  int table_pages, n_seq;
  int kv_blocks;              // the kernel's: blocks of the grid that take k and v
  int by_token;               // slots of sequences by their tokens (else by 16 of them)
  Divisor by_Hkv2;
};

#ifdef __CUDACC__
// Exponent of a scale; whatever else a damaged cache holds becomes one of the range
__device__ __forceinline__ int scale_exp(float s) {
  const int e = (int)((__float_as_uint(s) >> 23) & 255) - 127;
  return e < kScaleMin ? kScaleMin : e > kScaleMax ? kScaleMax : e;
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
#endif

// Barriers that are made to wait for an arrival that never comes, in tests only
// (moe_debug_attn_wait_timeout): their arrival count, a kernel argument, is one
// too many
enum Hold {
  kHoldNone, kHoldDecode,
  kHoldKeys, kHoldStage, kHoldQuery, kHoldS, kHoldP, kHoldO, kHoldHalf, kHoldTurn, kHoldItem, kHoldNext,    // attn_tc.cu
  kHolds
};

// One attention call.  Packed keys: k, v, kv_starts.  Paged: k_cache,
// v_cache, page_table, kv_lens.  Decode is n_seq rows of one token each
// (q_starts null) with an optional shared prefix.
struct AttnArgs {
  Heads q, k, v;
  const uint16_t* k_cache;    // (the cache in 8 bits: codes, with `scales`)
  const uint16_t* v_cache;
  const float* scales;        // null: k_cache and v_cache hold elements of the call's type
  const int32_t* page_table;  // [n_seq, table_pages], null when packed
  const int32_t* prefix_table;
  const int32_t* q_starts;
  const int32_t* kv_starts;
  const int32_t* kv_lens;
  int table_pages, pages, page_shift;
  int prefix_len;
  int n_seq, T, Tk, Hq, Hkv, D, f16, causal;
  float scale;
  uint16_t* out;              // [T, Hq, D]
  float* lse;                 // [T, Hq] or null
  int hold;                   // Hold
};

cudaError_t launch_rope_append(const RopeArgs& a, void* ws, int num_sms, cudaStream_t stream);
cudaError_t launch_rope_append_fp8(const RopeFp8Args& a, void* ws, int num_sms, cudaStream_t stream);

// attn_weights.cu -- attention weight of every key
struct WeightArgs {
  Heads q;
  const uint16_t* k_cache;    // [pages, Hkv, page_size, D]
  const int32_t* page_table;  // [n_seq, table_pages]
  const int32_t* q_starts;
  const int32_t* kv_lens;
  int table_pages, pages, page_shift;
  int n_seq, T, Hq, Hkv, D, f16, causal;
  float c;                    // scale log2 e
  const float* lse;           // [T, Hq]
  float* weights;             // [n_seq, Hkv, capacity]
  int capacity;
  Divisor by_G;
  int hold;                   // Hold
};
cudaError_t launch_attn_weights_tc(const WeightArgs& a, void* ws, int num_sms, cudaStream_t stream);
cudaError_t launch_attn_weights(const WeightArgs& a, void* ws, int num_sms, cudaStream_t stream);

// kv_evict.cu
struct EvictArgs {
  uint16_t* k_cache;          // [pages, Hkv, page_size, D]
  uint16_t* v_cache;
  const int32_t* page_table;  // [n_seq, table_pages]
  const int32_t* out_table;   // [n_seq, out_pages]
  const int32_t* kv_lens;
  const float* weights;       // [n_seq, Hkv, capacity]
  int table_pages, out_pages, pages, page_shift, capacity;
  int n_seq, Hkv, D;
  int budget, first, last;
  int32_t* new_lens;          // [n_seq]
  float* new_weights;         // [n_seq, Hkv, budget]
  int32_t* kept;              // [n_seq, Hkv, budget]
  Divisor by_Hkv, by_budget;
};
cudaError_t launch_kv_evict(const EvictArgs& a, void* ws, int num_sms, cudaStream_t stream);

// attn_tc.cu -- tiles of 128 rows (tt tokens x G heads), two per block; slots:
// tile slots of the batch (see find_seq)
struct TcPlan {
  int tt, slots;
};
inline TcPlan tc_plan(const AttnArgs& a) {
  const int tt = 128 / (a.Hq / a.Hkv), per = 2 * tt;
  return TcPlan{tt, a.q_starts ? a.T / per + a.n_seq : (a.T + per - 1) / per};
}
// Parts that a call splits each row's keys into (1: none, the result is final)
constexpr int kBlocksPerSplit = 4;
// A shared prefix leaves this share of the SMs to the rows' own keys, which are
// read meanwhile (64 sequences with 50 to 700 keys of their own after 16,384
// shared ones: 41 -> 33.4 us when it was done, now 29.7; after 512 26.5 -> 21.5,
// now 20.1; after 65,536 71 -> 73, now 68.0)
constexpr int kOwnShare = 6;
int tc_splits(const AttnArgs& a, int num_sms);
int tc_items(const AttnArgs& a, int splits);      // blocks of the grid; -1: too many
cudaError_t launch_attn_tc(const AttnArgs& a, int splits, float* part_o, float* part_lse, const Report& rep,
                           cudaStream_t stream);

// attn_decode.cu -- one token per sequence.  Parts of rows in the workspace:
// per row (tc_*: `splits` parts of the prefix [splits, T * Hq], then the row's
// own keys, row_*, null without a prefix), per block (two slots of 16 rows: a
// unit that began in an earlier block, and one that goes on in the next), the
// unit that each block's range ends in, {sequence, unit, blocks from this one
// on, 0} (0 blocks: none); with a prefix instead, for every unit, {blocks that
// hold its keys (one: the parts are in row order), the first of them}.
struct DecodeParts {
  float* tc_o;
  float* tc_lse;
  float* row_o;
  float* row_lse;
  float* slot_o;
  float* slot_lse;
  int4* tail;
  int2* held;
};
// A unit costs its warp about as much as one 16-key slice besides its slices
// (queries, the end of the softmax): 64 sequences of 1 to 8192 keys
constexpr int kUnitCost = 1;
// The line of all units' places, cut into ranges for the warps of as many
// blocks as have a place for each of their eight warps (up to the grid).  Its
// length is below 2^31 (decode_fits), which keeps the start of the kernel free
// of 64-bit divisions: code that runs once is fetched from L2 as it runs.
// With a shared prefix the first `few` blocks run beside its kernel, and their
// warps take up to `head` places, what they get through meanwhile; the others
// come after it and share the rest.
struct Line {
  int few, head;       // leading blocks and their places per warp (0: none)
  int each;            // places per warp of the others; the first `more` warps have one more
  int blocks, more;
  __host__ __device__ Line(int total, int grid, int few_, int head_) : few(few_), head(head_) {
    if (few > 0 && total / (8 * few) < head) grid = few;       // the leading blocks are enough
    if (few == 0 || grid == few) few = head = 0;
    const int rest = total - few * head * 8;
    const int n = rest / 8 + (rest % 8 != 0), most = grid - few;
    const int own = n < 1 ? 1 : n < most ? n : most;
    blocks = few + own;
    each = rest / (own * 8);
    more = rest - each * (own * 8);
  }
  // first place of warp g (of all blocks')
  __host__ __device__ int at(int g) const {
    const int i = g - few * 8;
    return i < 0 ? g * head : few * 8 * head + each * i + (i < more ? i : more);
  }
  // block of a place
  __host__ __device__ int block_of(int place) const {
    const int p = place - few * 8 * head, cut = (each + 1) * more;
    if (p < 0) return place / (8 * head);
    return few + (p < cut ? p / (each + 1) : more + (p - cut) / each) / 8;
  }
};
// The decode kernel beside that of a shared prefix: blocks that find room while
// it runs, and the places that each of their warps gets through: an SM reads
// ~100 GB/s by itself, and the other kernel takes ~1.6 us per 128 keys of its
// longest part and 8 us besides.  (With all blocks alike, the second round of
// them cost more than the first saved: 16,384 shared keys before 1 to 8192 own
// ones 67 us, this way 45, one kernel after the other 53; now 42.8.)
constexpr int kHeadFixed = 5, kHeadPerBlock = 3;
struct Beside {
  bool prefix;
  int few, head;
};
// The leading blocks' places with codes: what they get through beside the prefix's
// kernel and then the same share as the others, so that a short prefix, whose
// kernel leaves almost every SM free, does not leave all else to the few blocks
// that come after it (2 sequences of 120,000 keys behind 200, 32/4 heads of 128: 68
// us; the 16-bit cache's call, which goes without, 580).
__host__ __device__ inline int beside_head(int total, int grid, int few, int head) {
  const int rest = total / 8 - few * head;
  return rest > 0 ? head + rest / grid : head;
}
// Units of at most 16 heads per key-value head
inline int decode_chunks(const AttnArgs& a) { return (a.Hq / a.Hkv + 15) / 16; }
// The longest line that the page table allows
inline bool decode_fits(const AttnArgs& a) {
  const long long slices = ((((long long)a.table_pages << a.page_shift) + 15) / 16 + kUnitCost) * a.Hkv * decode_chunks(a);
  return slices < (1ll << 31) && slices * a.n_seq < (1ll << 31);
}
cudaError_t launch_attn_decode(const AttnArgs& a, const Beside& beside, const DecodeParts& p, const Report& rep,
                               int num_sms, cudaStream_t stream);

// attn_merge.cu -- joins the parts of every row (decode_grid 0: prefill)
cudaError_t launch_attn_merge(const AttnArgs& a, int splits, const DecodeParts& p, int decode_grid,
                              cudaStream_t stream);

}  // namespace attn
}  // namespace moe
