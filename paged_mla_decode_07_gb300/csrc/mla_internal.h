// Internal definitions shared by the libmla translation units (host API and
// kernels).  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <string>

#include "../../include/mla.h"

namespace mla {

constexpr int kDqk = 576;          // latent (512 NoPE) + 64 RoPE dims per token
constexpr int kDv = 512;           // value dims = first 512 key dims
constexpr int kChunk = 64;         // dims per 128-byte swizzle atom row (bf16)
constexpr int kNumChunks = 9;      // 576 / 64
constexpr int kPageSize = 64;      // tokens per page
constexpr int kTileTokens = 64;    // tokens per KV tile (one page) = MMA M of S^T = K Q^T
constexpr int kFp8RowBytes = 656;  // 512 e4m3 + 4 fp32 scales + 64 bf16
constexpr int kFp8ScaleOffset = 512;
constexpr int kFp8RopeOffset = 528;
constexpr int kSchedInts = 8;      // ints per schedule record

// Schedule record of one part (a group of `row_groups` CTAs that walk the
// same tiles, one CTA per row group):
//   [0] first problem  [1] first tile in it  [2] last problem (inclusive bound)
//   [3] end tile in the last problem (exclusive)  [4] split index of the
//   part's piece of its first problem  [5] number of parts the schedule was
//   cut into  [6] geometry tag of the decode it was made for  [7] unused (0)
// The decode kernel compares [5] and [6] of record 0 with its own launch
// before it reads any other record, so a schedule made for another
// configuration (or another device) is reported, never followed.
enum SchedField { kSchedP0 = 0, kSchedT0 = 1, kSchedP1 = 2, kSchedT1 = 3, kSchedSplit0 = 4, kSchedParts = 5,
                  kSchedTag = 6 };

constexpr int kMaxPages = ((1ll << 31) - 1) / kPageSize;  // slots are int32
constexpr int kMaxProblems = 16384;    // metadata kernel keeps per-problem prefix sums in smem

// Number of tiles of problem p: dense covers the cached tokens [0, seqlen),
// sparse covers the topk index slots of the query token.  Tiles are 64
// tokens (one page) for the single-CTA kernel and 128 (two pages, one per
// CTA) for the CTA-pair kernel.
__host__ __device__ inline int problem_tiles(const int32_t* cache_seqlens, int p, int s_q, int topk,
                                             int tile_tokens = kTileTokens) {
  if (topk > 0) return (topk + tile_tokens - 1) / tile_tokens;
  int L = cache_seqlens[p];
  return L > 0 ? (L + tile_tokens - 1) / tile_tokens : 0;
}

// Pages a windowed problem reads.  Query token i sits at position L - s_q + i
// and sees the first `sinks` keys and the last `window` up to its own, so all
// query tokens together see [0, sinks) and [L - s_q - window + 1, L): the
// first `head` pages, then those from page head + skip on (one run when the
// two touch).  Page i of the walk is page i, or i + skip from `head` on.  Of
// the pages past the `cols` columns of the block table a walk has one, whose
// lookup reports them: a length says nothing about the memory behind it.
struct KeyWalk {
  int pages, head, skip;
  __host__ __device__ int page(int i) const { return i < head ? i : i + skip; }
};
// Pages of L keys, at most one past the table.
__host__ __device__ inline int pages_of(int L, int cols) {
  if (L <= 0) return 0;
  const int n = (L - 1) / kPageSize + 1;
  return n <= cols ? n : cols + 1;
}
__host__ __device__ inline KeyWalk key_walk(int L, int s_q, int window, int sinks, int cols) {
  if (L <= 0) return KeyWalk{0, 0, 0};
  const int first = L - s_q - window + 1;  // > -2^31: window is at most 2^30, s_q at most 1024
  const int head = pages_of(sinks < L ? sinks : L, cols), w0 = first / kPageSize;
  if (first <= 0 || w0 <= head || head > cols) {
    const int n = pages_of(L, cols);
    return KeyWalk{n, n, 0};
  }
  const int total = (L - 1) / kPageSize + 1, end = (w0 > cols ? w0 : cols) + 1;
  return KeyWalk{head + (total < end ? total : end) - w0, head, w0 - head};
}
// Whether some query token of the element sees key t (t < L).
__host__ __device__ inline bool key_in_walk(int t, int L, int s_q, int window, int sinks) {
  return t < sinks || t > L - s_q - window;
}
constexpr int kMaxCluster = 8;       // CTAs of a cluster that share a windowed problem
constexpr int kMaxWindow = 1 << 30;  // larger windows see every key a cache can hold, as this one does

// Rows per CTA for a problem with `rows` query rows sharing one key set.
inline int rows_per_cta(int rows) { return rows > 32 ? 64 : (rows > 16 ? 32 : 16); }

struct Geometry {
  int num_problems;  // dense: batch; sparse: batch * s_q
  int rows;          // query rows per problem: dense s_q*h_q; sparse h_q
  int rpc;           // rows per CTA (16, 32, 64)
  int row_groups;    // ceil(rows / rpc)
  int num_parts;     // schedule parts (each = row_groups CTAs)
  int sm_count;
  int mode;          // decode kernel mode: 0 dense bf16, 1 sparse FP8, 2 dense FP8, 3 sparse bf16 rows, 4 and 5
                     // windowed 0 and 2, 6 shared prefix on CTA pairs, 7 windowed, operands in
                     // registers, 8 windowed over FP4 rows
  int pair;          // 1: CTA-pair kernel (128 rows and 128-token tiles per pair), 0: one CTA per row group
  int tile_tokens;   // tokens per schedule tile (64, or 128 for the pair kernel)
  int tile_cost;     // schedule cost of one tile (quarter units of a 64-token bf16 tile)
  int overhead;      // schedule cost of starting a problem segment (same units)
  int tag;           // geometry tag written into the schedule records
};

struct DecodeParams {
  const int32_t* block_table;
  const int32_t* cache_seqlens;
  const int32_t* indices;
  const int32_t* sched;
  const int32_t* num_splits;
  const uint8_t* kv_fp8;      // sparse: raw FP8 cache
  void* out;                  // bf16 [num_problems * rows, 512]
  float* lse;                 // [num_problems * rows]
  float* o_accum;             // [slots, rows, 512]
  float* lse_accum;           // [slots, rows]
  uint32_t* status;
  uint64_t timeout_ns;
  int batch, s_q, h_q, topk;
  int num_pages, block_table_stride;
  int num_problems, rows, row_groups, num_parts;
  int max_slots;              // partial-result slots the workspace holds
  int is_causal;
  int evict_first;
  int sched_tag;              // expected kSchedTag of the schedule records
  int debug_stall;            // test hook: the softmax role waits on a barrier nothing completes
  int flat_rows;              // > 0: sparse over an unpaged KV of this many rows (index = row; no
                              // block table or cache_seqlens); 0: paged cache
  const float* kv_scales;     // FP8 rows with one scale per token ([rows] fp32), else NULL
  const int32_t* topk_lengths;  // sparse: valid index slots per problem, else NULL
  int fp8_rope_off;           // byte offset of the RoPE dims in a row (FP8: 528, or 512 with kv_scales;
                              // bf16 rows: 1024)
  int rows16;                 // CTA-pair sparse decode: the rows are bf16 (1152 bytes, used as they
                              // are), 0: FP8 rows, dequantised

  int window, sinks;          // windowed modes: keys before a query token it sees, first keys that stay visible
  int cluster;                // > 0: each problem's pages over the CTAs of a cluster of this many (mla_cluster.cuh)
  int always_partial;         // every piece writes a partial result, the only piece of a problem too
  // windowed and shared-prefix decode make their schedules themselves (mla_schedule.cuh)
  int tile_cost, overhead;    // schedule costs
  int32_t* spans;             // [2 * problems] slot of the first piece, part of the last one

  // shared-prefix decode on CTA pairs: problem i is rows [128 i, 128 i + 128)
  // of the batch over the prefix and, with own_keys, then over the own keys of
  // each element that some of them belong to
  const int32_t* prefix_table;  // [prefix_pages]
  const int32_t* prefix_len;    // [1]
  int prefix_pages, total_rows, own_keys;

  float scale_log2;           // sm_scale * log2(e)
};

// What a schedule needs to know of the problems of windowed and shared-prefix decode.
struct SchedSpec {
  const int32_t* seqlens;     // [batch]
  int s_q;
  int window, sinks;          // window > 0: windowed problems
  int cols;                   // of the block table
  const int32_t* prefix_len;  // shared-prefix decode (see DecodeParams), else NULL
  int prefix_pages, rows, total_rows, own_keys;
};

// One kind of problems of a merge: where its pieces are and their partials.
struct MergeSide {
  const int32_t* spans;       // [2 * problems of this kind]
  const float* o;             // [slots, rows, 512]
  const float* lse;           // [slots, rows]
  int whole_base;             // slots before those of problems held whole; -1: these write the output themselves
};

// Merge of the partials of problems of `rows` query rows each (`own`) and,
// where an FP8 prefix has its own, of blocks of 128 rows (`prefix`).
struct MergeParams {
  MergeSide own, prefix;
  int has_prefix;
  int rows, problems, total_rows;
  void* out;
  float* lse;
};

struct CombineParams {
  const int32_t* num_splits;
  const int32_t* cache_seqlens;  // problems without tiles get out = 0, lse = -inf (sparse: unused)
  int s_q, topk;
  const float* o_accum;
  const float* lse_accum;
  void* out;
  float* lse;
  int num_problems, rows;
  int max_slots;
  uint32_t* status;
};

struct IndexParams {
  const float* q_scales;      // [num_tokens, h_idx]
  const float* weights;       // [num_tokens, h_idx]
  const int32_t* row_offsets; // [batch + 1]
  const float* k_scales;      // [num_pages * 64]
  const int32_t* block_table;
  const int32_t* cache_seqlens;
  float* scores;              // [num_tokens, width]
  uint32_t* status;
  uint64_t timeout_ns;
  int64_t width;              // block_table_stride * 64: the longest possible key range
  int batch, num_tokens, h_idx, max_new, n_box, num_pages, block_table_stride, relu, tiles_per_cta;
  uint32_t tmem_cols;         // two accumulator buffers of tmem_cols / 2 >= n_box columns
};

struct AssignPagesParams {
  const int32_t* cache_lengths;
  const int32_t* new_tokens;
  const int32_t* free_pages;
  const int32_t* free_cursor;
  int32_t* block_table;
  int32_t* cache_seqlens;  // NULL: not written by this launch (likewise the next three)
  int32_t* row_offsets;
  int32_t* slot_map;
  int32_t* next_cursor;
  uint32_t* status;
  int batch, num_free, block_table_stride, num_pages, num_tokens;
  int fill_table;          // 1: write the new block-table entries and the slots; 0: lengths and cursor only
};

// New tokens into cache rows by slot.
struct SlotStoreParams {
  const uint16_t* latent;  // bf16 [num_tokens, 512], rows latent_stride elements apart
  const uint16_t* rope;    // bf16 [num_tokens, 64], rows rope_stride elements apart
  const int32_t* slots;    // [num_tokens]
  uint8_t* kvcache;
  float* kv_scales;        // FP8 rows with one scale per token, else NULL
  uint32_t* status;
  int64_t latent_stride, rope_stride;
  int num_tokens, num_slots;
  int is_fp8;
  int is_fp4;              // FP4 rows (is_fp8 is 0)
};

// Cached tokens into packed bf16 rows.
struct CacheLoadParams {
  const uint8_t* kvcache;
  const float* kv_scales;      // FP8 rows with one scale per token, else NULL
  const int32_t* block_table;
  const int32_t* starts;       // [batch] first position of each request, or NULL: 0
  const int32_t* row_offsets;  // [batch + 1]
  uint8_t* out;                // bf16 [num_tokens, 576]
  uint32_t* status;
  int batch, block_table_stride, num_pages, num_tokens;
  int format;                  // mla_cache_format
};

// Attention over packed prompts.  The workspace: a counter, the number of blocks,
// and the list of blocks (8 ints each, 5 of them used); without a plan and with
// splits, the items (4 ints each) and the partial results.
constexpr int kPromptBlock = 256;  // query rows of a block
constexpr int kPromptCounter = 0, kPromptBlocks = 1, kPromptList = 64, kPromptEntryInts = 8;
struct PromptParams {
  const int32_t* q_offsets;  // [batch + 1]
  const int32_t* k_offsets;  // [batch + 1]
  int32_t* plan;             // workspace
  void* out;                 // bf16 [num_q, h_q, 128]
  float* lse;                // [num_q, h_q]
  uint32_t* status;
  uint64_t timeout_ns;
  int batch, num_q, num_k, h_q, h_kv;
  int max_blocks;            // blocks that the list has room for: as many as non-decreasing offsets can name
  int planned;               // 1: items by the plan; 0: item i belongs to CTAs i * splits ..
  int splits;                // CTAs that share an item's key tiles (1 with a plan)
  float* o_part;             // their results, [items * splits][256 rows][128]
  float* lse_part;           // [items * splits][256 rows]
  int causal, debug_stall;
  float scale_log2;
};

// Lets launches of a kernel whose shared memory varies from call to call have
// `bytes` of it beside the kernel's own (at most `own`).  48 KB in all need no
// leave.  The limit belongs to the kernel, not to the launch, and another host
// thread may set it between here and the launch: so every call sets the same
// one, the most a block can have.
template <class Kernel>
cudaError_t allow_dynamic_smem(Kernel* kernel, size_t bytes, size_t own) {
  constexpr size_t kFree = 48 * 1024, kMost = 227 * 1024;
  if (bytes + own <= kFree) return cudaSuccess;
  if (bytes + own > kMost) return cudaErrorInvalidValue;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMost - own));
}

// What a kernel that hands registers from warp to warp was compiled with, and what
// its split is for (setmaxnreg waits for ever for more than there are).  Read, and the
// kernel's shared memory allowed, once per device, before its first launch there.
struct KernelRegs {
  const char* kernel;
  int have, want;
};

// Kernel launchers (defined in the .cu files); return a CUDA error code.
cudaError_t launch_metadata(const int32_t* cache_seqlens, int s_q, int topk, const Geometry& g, int32_t* sched,
                            int32_t* num_splits, cudaStream_t stream);
// Windowed decode at 16 query rows per CTA on register-level matrix instructions (mla_decode_rows.cu)
// (tm_kv: bf16 rows alone)
cudaError_t launch_decode_rows(const CUtensorMap& tm_kv, const void* q, const DecodeParams& p, bool is_fp8,
                               cudaStream_t stream);
// Windowed decode over FP4 rows (mla_decode_fp4.cu)
// (tm_codes: codes and scales of a page as one box, tm_rope: its RoPE values; rpc: 16 or 32 rows per CTA)
// (the current device has had ready_decode_fp4)
cudaError_t launch_decode_fp4(const CUtensorMap& tm_codes, const CUtensorMap& tm_rope, const void* q, const DecodeParams& p,
                              int rpc, cudaStream_t stream);
cudaError_t ready_decode_fp4(int rpc, KernelRegs* regs);
// mode: 0 dense bf16 cache, 1 sparse FP8 cache, 2 dense FP8 cache, 3 sparse bf16 rows, 4 and 5 windowed dense
// over the bf16 and the FP8 cache
cudaError_t launch_decode(const CUtensorMap& tm_q, const CUtensorMap& tm_kv, const DecodeParams& p, int rpc,
                          int mode, cudaStream_t stream);
// CTA pairs the pair decode kernel can keep resident at once on the current
// device (0 if the query fails)
int pair_cluster_capacity();
// CTA-pair decode for problems of more than 64 rows: dense over the bf16 cache
// (tm_q, tm_ks, tm_kv: chunk-major maps with boxes of 9 chunks (Q), 3 and 2
// chunks (cache)) or sparse over the FP8 cache (tm_q as before, tm_ks: the
// FP8 rows as 128-byte boxes of one row for row gathers, tm_kv unused)
cudaError_t launch_decode_pair(const CUtensorMap& tm_q, const CUtensorMap& tm_ks, const CUtensorMap& tm_kv,
                               const DecodeParams& p, bool sparse, cudaStream_t stream);
// The same kernel, windowed or over a shared prefix and the elements' own keys (bf16 rows)
cudaError_t launch_window_pair(const CUtensorMap& tm_q, const CUtensorMap& tm_ks, const CUtensorMap& tm_kv,
                               const DecodeParams& p, cudaStream_t stream);
cudaError_t launch_prefix_pair(const CUtensorMap& tm_q, const CUtensorMap& tm_ks, const CUtensorMap& tm_kv,
                               const DecodeParams& p, cudaStream_t stream);
// FP8 prefix rows to bf16 rows in `rows` (page i of the prefix at rows + 64 i),
// `table[i]` = i or -1 for an unusable page
cudaError_t launch_prefix_rows(const uint8_t* kvcache, const float* kv_scales, const int32_t* prefix_table,
                               const int32_t* prefix_len, int prefix_pages, int num_pages, void* rows, int32_t* table,
                               uint32_t* status, int sm_count, cudaStream_t stream);
cudaError_t launch_combine(const CombineParams& p, cudaStream_t stream, bool pdl);
cudaError_t launch_merge(const MergeParams& p, cudaStream_t stream);
// Clusters of `size` single-CTA windowed kernels that are resident at once
int window_cluster_capacity(int size);
cudaError_t launch_fp8_cache_store(const uint16_t* x, int num_tokens, const int32_t* row_offsets,
                                   const int32_t* cache_lengths, int batch, const int32_t* block_table,
                                   int block_table_stride, uint8_t* kvcache, int num_pages, uint32_t* status,
                                   int sm_count, cudaStream_t stream);
cudaError_t launch_slot_store(const SlotStoreParams& p, int sm_count, cudaStream_t stream);
// (tm_q, tm_k_nope, tm_v: boxes of 64 values of one head of 128 rows; tm_k_rope: of 128 rows)
// (the current device has had ready_prompt)
cudaError_t launch_prompt(const CUtensorMap& tm_q, const CUtensorMap& tm_k_nope, const CUtensorMap& tm_k_rope,
                          const CUtensorMap& tm_v, const PromptParams& p, int sm_count, cudaStream_t stream);
cudaError_t ready_prompt(KernelRegs* regs);
cudaError_t launch_cache_load(const CacheLoadParams& p, int sm_count, cudaStream_t stream);
// in_place: the lengths or the cursor are updated in the arrays they are read from
cudaError_t launch_assign_pages(const AssignPagesParams& p, bool in_place, int sm_count, cudaStream_t stream);
cudaError_t launch_index(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const IndexParams& p, int topk,
                         int32_t* out, cudaStream_t stream);
// Sets the thread-local message returned by mla_last_error().
void set_error_message(const std::string& msg);

}  // namespace mla
