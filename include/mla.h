/*
 * libmla — paged Multi-head Latent Attention (MLA) decode for GB300 (sm_103a).
 *
 * C ABI.  Plain pointers and sizes only; every pointer named "device" must
 * point to memory of the current CUDA device.  The library never allocates
 * device memory: the caller sizes buffers with mla_metadata_size() and
 * mla_workspace_size() and passes them in.  All work is enqueued on the
 * caller's stream and is asynchronous; host-detectable errors return at once
 * with no launch, and mla_last_error() then names the offending argument.
 *
 * The two compute calls follow the decode API described in "Why FlashMLA's
 * decode kernel reaches 660 TFLOPS" (usage section): a scheduling-metadata
 * call made once per decode step and reused by every layer, then one decode
 * call per layer that returns the attention output and its log-sum-exp.
 *
 * Shapes (one KV head; the MQA form of MLA from the Modular design-doc
 * overview, section 9 "Multi-Head Latent Attention": a query row is 576-wide,
 * keys are 576-wide and the value is the first 512 dims of the key):
 *   q             bf16  [batch, s_q, h_q, 576], contiguous
 *   kvcache dense bf16  [num_pages, page_size, 1, 576], contiguous
 *   kvcache fp8   uint8 [num_pages, page_size, 1, 656], contiguous; per token
 *                 bytes [0,512) float8_e4m3 codes of dims 0..511, [512,528)
 *                 four float32 scales (scale k covers dims [128k,128k+128)),
 *                 [528,656) 64 bf16 RoPE values (FlashMLA article, Design 2)
 *   block_table   int32 [batch, block_table_stride]; logical token t of
 *                 element b lives in page block_table[b][t / page_size],
 *                 slot t % page_size (Modular overview, section 4
 *                 "PagedAttention")
 *   cache_seqlens int32 [batch]
 *   indices       int32 [batch, s_q, topk] logical token ids (sparse mode);
 *                 ids outside [0, cache_seqlens[b]) — e.g. -1 — are skipped,
 *                 repeated ids count once per occurrence
 *   out           bf16  [batch, s_q, h_q, 512]
 *   lse           fp32  [batch, s_q, h_q], base 2: log2(sum_j exp(s_j))
 *
 * out = softmax(q K^T * sm_scale) V over the key set of each query row:
 * dense mode = tokens [0, seqlen) (with is_causal: [0, seqlen - s_q + i] for
 * query token i), sparse mode = the valid ids of indices[b, i, :].  A row
 * with an empty key set gets out = 0 and lse = -inf.
 *
 * Supported modes (page_size 64): dense or sparse (top-k), each over a bf16
 * cache or an FP8 cache (is_fp8 selects the format); an FP8 cache may also
 * hold 640-byte rows (codes + RoPE) with one float32 scale per token in a
 * separate array (kv_scales).  Other page sizes return MLA_ERR_UNSUPPORTED.
 */
#ifndef MLA_H_
#define MLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The caller's CUDA stream (a cudaStream_t / CUstream); NULL = legacy default stream. */
typedef struct CUstream_st* mla_stream_t;

typedef enum {
  MLA_OK = 0,
  MLA_ERR_INVALID_ARG = 1,    /* null pointer, bad size or alignment; see mla_last_error() */
  MLA_ERR_UNSUPPORTED = 2,    /* valid request outside the supported modes/shapes */
  MLA_ERR_WORKSPACE = 3,      /* workspace missing or smaller than mla_workspace_size() */
  MLA_ERR_CUDA = 4,           /* a CUDA runtime/driver call failed; message has the error */
  MLA_ERR_DEVICE_BOUNDS = 5,  /* device status: a block-table entry outside [0, num_pages), or no room */
  MLA_ERR_DEVICE_TIMEOUT = 6  /* device status: a bounded wait inside a kernel gave up */
} mla_status;

/* Device status bits, reported by mla_get_device_status(). */
#define MLA_DEVICE_BAD_PAGE 0x1u     /* a page id outside [0, num_pages) was skipped (token masked) */
#define MLA_DEVICE_TIMEOUT 0x2u      /* a pipeline wait exceeded its limit; results are invalid */
#define MLA_DEVICE_BAD_SCHEDULE 0x4u /* the schedule did not match the arguments; results invalid */
#define MLA_DEVICE_NO_ROOM 0x8u      /* mla_assign_pages ran out of free pages, table columns or slot entries */

/* ABI version of this header (incremented on incompatible change). */
#define MLA_ABI_VERSION 3
int mla_abi_version(void);

/* A decode configuration is the tuple (batch, h_q, s_q, topk, is_fp8), in the
 * order of the FlashMLA article's get_mla_metadata(cache_seqlens, ..., h_q,
 * is_fp8, topk) (usage section); topk = 0 selects dense mode, is_fp8 = 1 an
 * FP8 cache.  The three calls below and mla_decode must see the same tuple:
 * the schedule depends on it (rows per CTA, the kernel mode and the cost of a
 * tile in that mode) and on the current device's SM count, so a schedule
 * belongs to one configuration on one device. */

/* Sizes of the two metadata arrays for a decode configuration on the
 * current device (int32 element counts).  sched has one 8-int record per
 * scheduled work part; num_splits has one entry per problem plus one
 * (problem = batch element in dense mode, (batch element, query token) pair
 * in sparse mode). */
mla_status mla_metadata_size(int batch, int h_q, int s_q, int topk, int is_fp8, int* sched_elems,
                             int* num_splits_elems);

/* Scratch bytes that mla_decode needs for split-KV partial results
 * (fp32 partial outputs and their log-sum-exps): min(2 * parts,
 * problems + parts) slots of rows x 513 floats, bounded by the part count
 * whatever the batch size. */
mla_status mla_workspace_size(int batch, int h_q, int s_q, int topk, int is_fp8, size_t* bytes);

/* (1) Tile schedule for one decode step ("get_mla_metadata").
 * cache_seqlens: device int32 [batch]; sched, num_splits: device int32
 * buffers of the sizes above, written on `stream`.  The work of all problems
 * (64-token tiles of their key ranges, each tile weighted by the cost of its
 * mode, FP8 tiles 1.5 times a bf16 tile, plus a fixed start-up cost per
 * problem segment) is divided into contiguous ranges of near-equal cost,
 * one per part; num_splits holds the exclusive prefix sum of the split-KV
 * partial-result slots of each problem: as many as the parts touching it
 * when there are two or more, none when one part covers it (that part writes
 * the output directly).  Every sched record also holds the part count and a
 * tag of the configuration; mla_decode checks both on the device against its
 * own and, on a mismatch, sets MLA_DEVICE_BAD_SCHEDULE and computes nothing
 * (it reads only the first record before that check).  Reusable by every
 * layer of the step as long as cache_seqlens and the configuration are
 * unchanged. */
mla_status mla_get_metadata(const int32_t* cache_seqlens, int batch, int h_q, int s_q, int topk, int is_fp8,
                            int32_t* sched, int32_t* num_splits, mla_stream_t stream);

/* Arguments of mla_decode.  Pointers are device pointers unless noted. */
typedef struct {
  const void* q;                  /* bf16 [batch, s_q, h_q, 576] */
  int batch, s_q, h_q;
  const void* kvcache;            /* bf16 [num_pages,64,1,576], uint8 [num_pages,64,1,656], or with
                                     kv_scales uint8 [num_pages,64,1,640] */
  int num_pages, page_size;       /* page_size must be 64 */
  const int32_t* block_table;     /* int32 [batch, block_table_stride] */
  int block_table_stride;         /* >= ceil(max seqlen / page_size) */
  const int32_t* cache_seqlens;   /* int32 [batch] */
  float sm_scale;                 /* softmax scale applied to q.k */
  int is_causal;                  /* dense only: query token i sees keys <= seqlen - s_q + i */
  int is_fp8;                     /* 1: FP8 cache rows (656 bytes; 640 with kv_scales), 0: bf16
                                     576-value rows (either mode) */
  const int32_t* indices;         /* sparse: int32 [batch, s_q, topk]; NULL for dense */
  int topk;                       /* 0 for dense */
  const int32_t* sched;           /* from mla_get_metadata with the same batch/h_q/s_q/topk/is_fp8 */
  const int32_t* num_splits;
  void* workspace;                /* >= mla_workspace_size() bytes, 256-byte aligned */
  size_t workspace_bytes;
  void* out;                      /* bf16 [batch, s_q, h_q, 512] */
  float* lse;                     /* fp32 [batch, s_q, h_q] */
  /* ABI version 2 (zero when unused): */
  const float* kv_scales;         /* FP8 cache with one scale per token (MAX kernels summary, MLA section:
                                     the scaled decode's per-token KV scales and 640-byte FP8 + BF16 rows):
                                     fp32 [num_pages, 64]; the cache rows are then uint8 [.., 640] = 512
                                     E4M3 codes + 64 bf16 RoPE values, K[d] = bf16_rn(e4m3 * scale) for
                                     d < 512.  NULL: 656-byte rows with four scales each. */
  const int32_t* topk_lengths;    /* sparse, optional: int32 [batch, s_q]; row (b, i) reads only its first
                                     topk_lengths[b, i] index slots (clamped to [0, topk]); NULL: all topk
                                     slots, -1 marking unused ones */
} mla_decode_args;

/* (2) Decode ("flash_mla_with_kvcache"): split-KV attention kernel followed
 * by a log-sum-exp combine of the split partials, both on `stream`.
 * Alignment: q, kvcache and out 16-byte aligned, lse, block_table and
 * kv_scales 4-byte aligned, workspace 256-byte aligned.  Every wait inside
 * the kernels is bounded (2 s by default; the environment variable
 * MLA_WATCHDOG_NS sets another limit in nanoseconds): a wait that runs out
 * sets MLA_DEVICE_TIMEOUT and the kernel returns. */
mla_status mla_decode(const mla_decode_args* args, mla_stream_t stream);

/* Decode without any caller scratch, for callers that cannot allocate device
 * memory when they decode (for example code inside a runtime or plugin host
 * that owns no CUDA memory pool, or a latency-critical path where cudaMalloc
 * is not allowed).  The pages describe no such entry point; it is an addition
 * of this library.  Same arguments and results as mla_decode, except that
 * workspace/workspace_bytes are ignored: the split-KV partials go to a fixed
 * 32 MiB array in the library's device memory, which every GPU that loads
 * this part of the library keeps until exit.  A decode whose scratch (see
 * mla_workspace_size) exceeds 32 MiB returns MLA_ERR_WORKSPACE without
 * launching anything.  The first call on a device looks the array up (once
 * per device) and should come before any stream capture.  All calls share the
 * array, so calls that overlap on the GPU race; serialise them.  Nothing in
 * the array needs to start at zero. */
mla_status mla_decode_noalloc(const mla_decode_args* args, mla_stream_t stream);

/* FP8 cache write: quantise new tokens into the 656-byte FP8 cache row and
 * store them through the block table (the step before a sparse FP8 decode).
 *
 * Row format ("Why FlashMLA's decode kernel reaches 660 TFLOPS", Design 2):
 * dims 0..511 as float8_e4m3 codes in four 1 x 128 tiles, each tile with one
 * float32 scale = amax / 448 (1 for an all-zero tile), code = E4M3 of
 * x / scale (float32 division) rounded to nearest even and saturated at 448;
 * bytes [512, 528) the four scales; bytes [528, 656) dims 512..575 as bf16.
 * Placement (MAX kernels summary, KV-cache store section): the new tokens of
 * batch element b are rows input_row_offsets[b] .. input_row_offsets[b+1]-1
 * of x and go to positions cache_lengths[b] + i of element b, i.e. page
 * block_table[b * block_table_stride + pos / 64], slot pos % 64.
 *
 *   x                 bf16 [num_tokens, 576], device, 16-byte aligned
 *   input_row_offsets int32 [batch + 1], device, non-decreasing, from 0 to num_tokens
 *   cache_lengths     int32 [batch], device: tokens already cached per element
 *   block_table       int32 [batch, block_table_stride], device
 *   kvcache           uint8 [num_pages, 64, 1, 656], device, 16-byte aligned; written
 * The caller owns all memory; the call is asynchronous on `stream`.  A token
 * whose page entry lies past block_table_stride or outside [0, num_pages) is
 * not written and sets MLA_DEVICE_BAD_PAGE in the device status word.  Host-
 * side argument errors return MLA_ERR_INVALID_ARG / MLA_ERR_UNSUPPORTED
 * (page_size != 64) without launching.  num_tokens == 0 launches nothing. */
mla_status mla_fp8_cache_store(const void* x, int num_tokens, const int32_t* input_row_offsets,
                               const int32_t* cache_lengths, int batch, const int32_t* block_table,
                               int block_table_stride, void* kvcache, int num_pages, int page_size,
                               mla_stream_t stream);

/* Pages and slots of one step's new tokens: the block table and the slot map
 * that the cache writes and the decode calls of the step use, built on the
 * device from the request lengths.
 *
 * Request b has max(cache_lengths[b], 0) cached tokens in the pages of its
 * block-table row and receives max(new_tokens[b], 0) more.  Pages it lacks
 * are taken from free_pages, from entry *free_cursor on, in the order of the
 * requests; they go to the next columns of its row (all other entries of
 * block_table are left as they are).  Written besides:
 *   cache_seqlens[b] = cached + new tokens   (the lengths decode takes)
 *   row_offsets[b]   = new tokens of the requests before b; row_offsets[batch] all
 *   slot_map[t]      = page * 64 + position % 64 of new token t (tokens in the
 *                      order of row_offsets), -1 for t past the last token
 *   *next_cursor     = *free_cursor + the pages taken
 * cache_seqlens may be cache_lengths itself and next_cursor free_cursor
 * itself (a decode loop recorded as a graph advances both in place); any
 * other overlap of an output is refused.
 *
 * A page that the free list or the table row has no room for gets table entry
 * -1 (if the row has the column) and its tokens slot -1; a token past
 * num_tokens gets no slot; either sets MLA_DEVICE_NO_ROOM.  A page id outside
 * [0, num_pages) gives its tokens slot -1 and sets MLA_DEVICE_BAD_PAGE.
 * The cursor is taken as clamped to [0, num_free].  Asynchronous on `stream`;
 * all memory is the caller's; batch at most 16384. */
typedef struct {
  const int32_t* cache_lengths;   /* int32 [batch] */
  const int32_t* new_tokens;      /* int32 [batch] */
  int batch;
  const int32_t* free_pages;      /* int32 [num_free], distinct page ids */
  int num_free;
  const int32_t* free_cursor;     /* int32 [1] */
  int32_t* block_table;           /* int32 [batch, block_table_stride], updated */
  int block_table_stride;
  int num_pages;                  /* pages of the cache */
  int num_tokens;                 /* entries of slot_map */
  int32_t* cache_seqlens;         /* out: int32 [batch] */
  int32_t* row_offsets;           /* out: int32 [batch + 1] */
  int32_t* slot_map;              /* out: int32 [num_tokens] */
  int32_t* next_cursor;           /* out: int32 [1] */
} mla_assign_pages_args;

mla_status mla_assign_pages(const mla_assign_pages_args* args, mla_stream_t stream);

/* Cache write through a slot map: token i, its 512 latent values and 64 RoPE
 * values from two row-strided tensors (rows of separate tensors, or slices of
 * one wider projection), goes to cache row slot_map[i] = page * 64 + slot.
 *
 * Row formats: is_fp8 = 0, bf16 rows of 576 values, copied; is_fp8 = 1, the
 * 656-byte rows of mla_fp8_cache_store, bit for bit as it writes them; with
 * kv_scales, 640-byte rows of 512 E4M3 codes and 64 bf16 RoPE values, with
 * scale = amax / 448 over the token's 512 latent values (1 for an all-zero
 * token) in kv_scales and code = E4M3 of x / scale (float32 division), rounded
 * to nearest even and saturated at 448.  (Of rows with a scale of 2^39 or more, a
 * latent value of 2^47.8, see mla_window_decode.)
 * A negative slot is padding and is skipped; a slot past the cache is not
 * written and sets MLA_DEVICE_BAD_PAGE.  Slots that are written must be
 * distinct: a row named twice may end up with bytes of either token.  Rows
 * that no slot names are left as they are.  Asynchronous on `stream`. */
typedef struct {
  const void* latent;             /* bf16 [num_tokens, 512], 16-byte aligned */
  int64_t latent_stride;          /* elements between rows: a multiple of 8 */
  const void* rope;               /* bf16 [num_tokens, 64], 16-byte aligned */
  int64_t rope_stride;            /* elements between rows: a multiple of 8 */
  const int32_t* slot_map;        /* int32 [num_tokens] */
  int num_tokens;                 /* 0: nothing is launched */
  void* kvcache;                  /* bf16 [num_pages,64,1,576], uint8 [num_pages,64,1,656 or 640], 16-byte aligned */
  int num_pages, page_size;       /* page_size must be 64 */
  int is_fp8;
  float* kv_scales;               /* fp32 [num_pages, 64] for 640-byte rows, else NULL */
} mla_cache_store_args;

mla_status mla_cache_store(const mla_cache_store_args* args, mla_stream_t stream);

/* FP4 cache rows: uint8 [num_pages, 64, 1, 400], per token 512 latent values
 * in 4 bits and 64 RoPE values in bf16.
 *   bytes [0, 256)    64 little-endian words of eight codes; word w holds dims
 *                     8 w .. 8 w + 7: bits 4 i .. 4 i + 2 are the magnitude of
 *                     dim i (0, 1/2, 1, 3/2, 2, 3, 4, 6: E2M1), bit 8 i + 7 the
 *                     sign of dim i and bit 8 i + 3 that of dim 4 + i (i < 4)
 *   bytes [256, 272)  16 scale bytes, one per 32 dims: 2^(byte - 127).  Bytes
 *                     are 114 to 140; others are read as the nearest of these
 *   bytes [272, 400)  64 bf16 RoPE values
 * value = code * scale, a bf16 number; every row's latent values are finite.
 *
 * mla_fp4_cache_store writes token i (as mla_cache_store does, with the same
 * rules for slots) with scale = 2^e, e the smallest integer with amax <= 6 * 2^e
 * over the 32 values, from -13 to 13, and code = E2M1 of x / scale, rounded to
 * nearest even and saturated at 6 (latents above 49152 are cut off there, those
 * of a block below 2^-15 become 0; NaN is stored as 6 * scale).  Normally
 * distributed latents come back with a relative error of 0.118 (root mean
 * square).  Asynchronous on `stream`. */
typedef struct {
  const void* latent;             /* bf16 [num_tokens, 512], 16-byte aligned */
  int64_t latent_stride;          /* elements between rows: a multiple of 8 */
  const void* rope;               /* bf16 [num_tokens, 64], 16-byte aligned */
  int64_t rope_stride;            /* elements between rows: a multiple of 8 */
  const int32_t* slot_map;        /* int32 [num_tokens] */
  int num_tokens;                 /* 0: nothing is launched */
  void* kvcache;                  /* uint8 [num_pages,64,1,400], 16-byte aligned */
  int num_pages, page_size;       /* page_size must be 64 */
} mla_fp4_cache_store_args;

mla_status mla_fp4_cache_store(const mla_fp4_cache_store_args* args, mla_stream_t stream);

/* Row formats of a cache. */
typedef enum {
  MLA_CACHE_BF16 = 0,       /* 576 bf16 values */
  MLA_CACHE_FP8 = 1,        /* 656 bytes, four scales */
  MLA_CACHE_FP8_TOKEN = 2,  /* 640 bytes, one scale per token in kv_scales */
  MLA_CACHE_FP4 = 3         /* 400 bytes, see mla_fp4_cache_store */
} mla_cache_format;

/* Reads cached tokens back as packed bf16 rows, as a chunked prefill needs them
 * for its up-projection: row t of out, row_offsets[b] <= t < row_offsets[b + 1],
 * is the token at position starts[b] + t - row_offsets[b] of request b, 512
 * latent and 64 RoPE values.  The values are those that the row stands for:
 * bf16 rows as they are, FP8 codes times their scale rounded to bf16, FP4
 * values exactly.  Rows of out from row_offsets[batch] on are left as they are;
 * offsets past num_tokens are cut off there.  A token whose page lies past
 * block_table_stride or outside [0, num_pages) becomes a row of zeros and sets
 * MLA_DEVICE_BAD_PAGE.  Asynchronous on `stream`. */
typedef struct {
  const void* kvcache;            /* as `format` says, 16-byte aligned */
  int num_pages, page_size;       /* page_size must be 64 */
  int format;                     /* mla_cache_format */
  const float* kv_scales;         /* fp32 [num_pages, 64] with MLA_CACHE_FP8_TOKEN, else NULL */
  const int32_t* block_table;     /* int32 [batch, block_table_stride] */
  int block_table_stride;
  int batch;
  const int32_t* starts;          /* int32 [batch], or NULL: every request from its first token on */
  const int32_t* row_offsets;     /* int32 [batch + 1], non-decreasing, from 0 */
  int num_tokens;                 /* rows of out; 0: nothing is launched */
  void* out;                      /* bf16 [num_tokens, 576], 16-byte aligned */
} mla_cache_load_args;

mla_status mla_cache_load(const mla_cache_load_args* args, mla_stream_t stream);

/* Windowed decode over FP4 rows: mla_window_decode's keys, masks and results
 * (a window of 2^30 or more sees every key: causal decode over the whole cache),
 * with its rules for missing pages and sizes.  Latent values and their products
 * with q are exact (q to 2^-21 of the largest value of its row), sums fp32, and
 * a probability is off by the larger of 2^-9 of itself and 2^-33 of the row's
 * largest (of n keys that far below it out may so lose n * 2^-33 of their mean
 * |v|; lse does not).  The RoPE values of a key that some query token sees must
 * be finite, or rows of its element are not.  A row of q that is not finite has
 * results that are not, other rows are as they would be.  All launches are made
 * on `stream` by the one call.
 * Rows are converted for every 32 of s_q * h_q: up to 64 of these the call is as
 * fast (to 4 %) as mla_window_decode over bf16 rows or faster (64 elements of 2048
 * to 16384 keys: 16 rows 73 us for 125, 32 rows 104 for 143, 64 rows 159 for 155),
 * with more it is slower (128 rows 293 for 185; 32 elements of 1001 to 8191 keys,
 * 128 rows 95 for 65); over FP8 rows the same calls take 121 to 402 us. */
typedef struct {
  const void* q;                  /* bf16 [batch, s_q, h_q, 576], 16-byte aligned */
  int batch, s_q, h_q;            /* s_q * h_q <= 1024 */
  const void* kvcache;            /* uint8 [num_pages,64,1,400], 16-byte aligned */
  int num_pages, page_size;       /* page_size must be 64 */
  const int32_t* block_table;     /* int32 [batch, block_table_stride] */
  int block_table_stride;
  const int32_t* cache_seqlens;   /* int32 [batch] */
  float sm_scale;
  int window;                     /* >= 1 */
  int sinks;                      /* >= 0 */
  void* workspace;                /* >= mla_fp4_decode_workspace_size() bytes, 256-byte aligned */
  size_t workspace_bytes;
  void* out;                      /* bf16 [batch, s_q, h_q, 512], 16-byte aligned */
  float* lse;                     /* fp32 [batch, s_q, h_q], base 2 */
} mla_fp4_decode_args;

mla_status mla_fp4_decode_workspace_size(int batch, int h_q, int s_q, size_t* bytes);
mla_status mla_fp4_decode(const mla_fp4_decode_args* args, mla_stream_t stream);

/* Attention over whole prompts, packed: the form of prefill before the
 * up-projections are absorbed.  Queries and keys are 192 wide, 128 values per
 * head and 64 RoPE values that all heads of a key share; values are 128 wide.
 *   out[i, h] = softmax(sm_scale * q[i, h] . (k_nope[t, h'], k_rope[t])) v[t, h'],
 *   h' = h / (h_q / h_kv)
 * Sequence b has query rows q_offsets[b] .. q_offsets[b + 1] (n of them) and key
 * rows k_offsets[b] .. k_offsets[b + 1] (m); either may be none.  With
 * is_causal, query row i of the sequence sees its first m - n + i + 1 keys (the
 * last query the last key: with context the queries are a prompt's last chunk;
 * m < n leaves the first rows without keys), else all m.  A row without keys
 * gets out = 0 and lse = -inf.  Rows of out and lse from q_offsets[batch] on are
 * left as they are.  Keys and values of other sequences may hold anything; a value
 * that is not finite shows in rows of its sequence.  Probabilities are rounded to
 * bf16, sums are fp32, lse is base 2 as in mla_decode.
 * All row and head strides are in elements and multiples of 8, so q, keys and
 * values may be slices (of one up-projection, of cache rows).  Offsets that
 * leave the rows are cut off there; results of offsets that decrease are
 * invalid, and set MLA_DEVICE_BAD_SCHEDULE where they name more blocks of 256
 * query rows than others could.
 * All launches are made on `stream` by the one call. */
typedef struct {
  const void* q;                  /* bf16 [num_q, h_q, 192], 16-byte aligned (as k_nope, k_rope and v) */
  int64_t q_stride, q_head_stride;
  int num_q, h_q;                 /* num_q = 0: nothing is launched; num_q, num_k <= 2^31 - 512 */
  const void* k_nope;             /* bf16 [num_k, h_kv, 128] */
  int64_t k_nope_stride, k_nope_head_stride;
  const void* k_rope;             /* bf16 [num_k, 64] */
  int64_t k_rope_stride;
  const void* v;                  /* bf16 [num_k, h_kv, 128] */
  int64_t v_stride, v_head_stride;
  int num_k, h_kv;                /* h_q a multiple of h_kv */
  const int32_t* q_offsets;       /* int32 [batch + 1], non-decreasing, from 0 */
  const int32_t* k_offsets;       /* int32 [batch + 1], non-decreasing, from 0 */
  int batch;
  float sm_scale;
  int is_causal;
  void* workspace;                /* >= mla_prompt_attention_workspace_size() bytes, 256-byte aligned */
  size_t workspace_bytes;
  void* out;                      /* bf16 [num_q, h_q, 128], 16-byte aligned */
  float* lse;                     /* fp32 [num_q, h_q], base 2 */
} mla_prompt_attention_args;

mla_status mla_prompt_attention_workspace_size(int num_q, int num_k, int h_q, int batch, size_t* bytes);
mla_status mla_prompt_attention(const mla_prompt_attention_args* args, mla_stream_t stream);

/* Sparse prefill ("flash_mla_sparse_fwd(q, kv, indices, sm_scale)" of the
 * FlashMLA article's usage section): token-level sparse attention with no
 * batch dimension and an unpaged bf16 KV with one head.  For query token i
 * and head h the rows kv[indices[i, k]] are gathered (ids outside [0, s_kv)
 * are skipped, a repeated id counts once per occurrence), logits
 * s_k = sm_scale * q[i, h] . kv[id_k], and
 *   out[i, h] = sum_k softmax(s)_k kv[id_k][0:512],   lse[i, h] = log2 sum_k e^{s_k}
 * (base-2 log-sum-exp of the natural logits; no valid id: out = 0,
 * lse = -inf).  The same computation as sparse decode with one batch element
 * whose cache is the KV itself; the library runs its decode kernels on
 * chunks of at most 16384 query tokens. */
typedef struct {
  const void* q;                  /* bf16 [s_q, h_q, 576], 16-byte aligned */
  int s_q, h_q;                   /* h_q <= 1024 */
  const void* kv;                 /* bf16 [s_kv, 576] (the single KV head squeezed out), 16-byte aligned */
  int s_kv;
  const int32_t* indices;         /* int32 [s_q, topk] */
  int topk;                       /* >= 1 */
  float sm_scale;
  void* workspace;                /* >= mla_sparse_prefill_workspace_size() bytes, 256-byte aligned */
  size_t workspace_bytes;
  void* out;                      /* bf16 [s_q, h_q, 512], 16-byte aligned */
  float* lse;                     /* fp32 [s_q, h_q] */
} mla_sparse_prefill_args;

/* Scratch bytes for mla_sparse_prefill: one chunk's schedule and split-KV
 * partials (independent of s_q beyond the first 16384 tokens). */
mla_status mla_sparse_prefill_workspace_size(int s_q, int h_q, int topk, size_t* bytes);

/* Asynchronous on `stream`; all pointers are device pointers owned by the
 * caller.  Host-side argument errors return without launching; device-side
 * problems set bits in the device status word (mla_get_device_status). */
mla_status mla_sparse_prefill(const mla_sparse_prefill_args* args, mla_stream_t stream);

/* Windowed decode: attention over the first `sinks` keys and the last
 * `window` keys of each element (sinks: first tokens that stay visible when
 * the window has moved past them).  Query token i of element b sits at
 * position P_i = cache_seqlens[b] - s_q + i and sees key t < cache_seqlens[b]
 * if t <= P_i and (t < sinks or t > P_i - window).  Results as mla_decode's;
 * a row that sees no key gets out = 0 and lse = -inf.  Only the pages that
 * hold keys some query token sees are read, so the others need no
 * block-table entry.  A key that no query token of its element sees may hold
 * anything; one that some of them see must be finite, or rows of its element
 * are not (those of other elements are).  Keys whose pages are missing from
 * the block table, or past its columns, are left out and set
 * MLA_DEVICE_BAD_PAGE.  batch * block_table_stride is at most 2^28.
 * FP8 caches: scales are positive.  With up to 16 query rows per element (s_q *
 * h_q; in calls of few pages with more), a value enters its sum as code * scale,
 * without the rounding to bf16 that it has in mla_decode (and as part of K), and
 * probability * scale is what is rounded to bf16.  That product is held at 2^80
 * times its value: an element that sees a key with a scale of 2^39 or more may
 * come out not finite.  Elements of at most 36 pages add what that rounding
 * left; an element's own pages alone decide on that.  Error against 64 bits,
 * relative, normal keys, at 1 / 16 / 36 / 37 / 66 / 200 pages: FP8 0.0022 /
 * 0.0020 / 0.0019 / 0.0022 / 0.0020 / 0.0018, bf16 0.0021 / 0.0020 / 0.0019 /
 * 0.0019 / 0.0018 / 0.0018 (0.0017 is the rounding of the result).
 * The attention kernel, which makes its schedule itself, and the merge of its
 * partial results are launched on `stream` by the one call. */
typedef struct {
  const void* q;                  /* bf16 [batch, s_q, h_q, 576], 16-byte aligned */
  int batch, s_q, h_q;            /* s_q * h_q <= 1024 */
  const void* kvcache;            /* as in mla_decode_args */
  int num_pages, page_size;       /* page_size must be 64 */
  const int32_t* block_table;     /* int32 [batch, block_table_stride] */
  int block_table_stride;
  const int32_t* cache_seqlens;   /* int32 [batch] */
  float sm_scale;
  int window;                     /* >= 1 */
  int sinks;                      /* >= 0 */
  int is_fp8;
  const float* kv_scales;         /* fp32 [num_pages, 64] for 640-byte FP8 rows, else NULL */
  void* workspace;                /* >= mla_window_decode_workspace_size() bytes, 256-byte aligned */
  size_t workspace_bytes;
  void* out;                      /* bf16 [batch, s_q, h_q, 512], 16-byte aligned */
  float* lse;                     /* fp32 [batch, s_q, h_q], base 2 */
} mla_window_decode_args;

mla_status mla_window_decode_workspace_size(int batch, int h_q, int s_q, int is_fp8, size_t* bytes);
mla_status mla_window_decode(const mla_window_decode_args* args, mla_stream_t stream);

/* Shared-prefix decode: a batch whose elements share their first tokens (one
 * system prompt, one document).  Every query row attends to the
 * *prefix_length tokens of prefix_table and to its element's own
 * cache_seqlens[b] tokens of block_table row b; with is_causal query token i
 * sees own keys <= cache_seqlens[b] - s_q + i (and always the whole prefix).
 * Results as mla_decode's over the two key sets in one softmax.  The prefix
 * is read and multiplied once for 128 query rows of the whole batch at a
 * time, whatever elements they belong to (calls of few pages: for 16 rows of
 * an element); with an FP8 cache it is turned into bf16 rows in the workspace
 * for that.  The prefix may end inside a page; own tokens start in pages of
 * their own.  Keys past a length may hold anything; keys that are not finite show in the rows that share them: all for
 * the prefix, the element's for own keys.  Missing pages, limits and FP8 caches as for
 * mla_window_decode (a prefix that is turned into bf16 rows has mla_decode's values).
 * The lengths are on the device, so the choice of the kernels and the FP8
 * workspace go by the widths of the tables.  Tables much wider than their keys
 * lose a small call its path (taken while prefix_table_len + block_table_stride
 * is at most 8 pages, over FP8 14, for each of the up to 8 CTAs that share an
 * element's pages): 6 x 16 rows behind 1999 keys take 17.8 us with 36 columns in
 * all and 21.8 to 22.4 with 68 to 1024, over FP8 20.9 with 96 and 34.7 with 516.
 * Each column of an FP8 prefix table is 73,728 bytes of workspace.  Give tables as wide as
 * the longest prefix and element.
 * All launches are made on `stream` by the one call. */
typedef struct {
  const void* q;                  /* bf16 [batch, s_q, h_q, 576], 16-byte aligned */
  int batch, s_q, h_q;            /* s_q * h_q <= 1024 */
  const void* kvcache;            /* as in mla_decode_args */
  int num_pages, page_size;       /* page_size must be 64 */
  const int32_t* prefix_table;    /* int32 [prefix_table_len]: page ids of the prefix */
  int prefix_table_len;
  const int32_t* prefix_length;   /* int32 [1], device: tokens of the prefix */
  const int32_t* block_table;     /* int32 [batch, block_table_stride]: pages of the own tokens */
  int block_table_stride;
  const int32_t* cache_seqlens;   /* int32 [batch]: own tokens */
  float sm_scale;
  int is_causal;
  int is_fp8;
  const float* kv_scales;         /* fp32 [num_pages, 64] for 640-byte FP8 rows, else NULL */
  void* workspace;                /* >= mla_shared_prefix_decode_workspace_size() bytes, 256-byte aligned */
  size_t workspace_bytes;
  void* out;                      /* bf16 [batch, s_q, h_q, 512], 16-byte aligned */
  float* lse;                     /* fp32 [batch, s_q, h_q], base 2 */
} mla_shared_prefix_decode_args;

mla_status mla_shared_prefix_decode_workspace_size(int batch, int h_q, int s_q, int prefix_table_len, int is_fp8,
                                                   size_t* bytes);
mla_status mla_shared_prefix_decode(const mla_shared_prefix_decode_args* args, mla_stream_t stream);

/* FP8 top-k indexer (MAX kernels summary, MLA indexing kernels:
 * mla_fp8_index_top_k): picks, per query token, the topk cached keys that
 * sparse attention will read.  The pages name its steps (FP8 scores with
 * scales, aggregation over the index heads, masking, int32 top-k with -1
 * fill) but give no formula; this library computes, for query row t of
 * element b (rows row_offsets[b] .. row_offsets[b+1]-1, the last n_b
 * positions of a cache of cache_seqlens[b] keys, so row j sees keys
 * s <= seqlen - n_b + j):
 *   score(t, s) = sum_h weights[t,h] * f(q_scales[t,h] * k_scales[s] * sum_d q[t,h,d] * k[s,d])
 * with E4M3 codes q, k (head dim 128), f = ReLU if relu != 0 else identity,
 * (q_scales and k_scales positive, as the amax / 448 quantiser makes them)
 * and writes the ids of the topk visible keys of largest score, in
 * descending score order (ties to the smaller id), -1 after the last visible
 * key.  Scores are computed in fp32 from the exact E4M3 products; keys whose
 * scores differ by less than that rounding may be ordered either way.  Key s
 * of element b is row block_table[b * block_table_stride + s / 64] * 64 + s % 64
 * of the key cache. */
typedef struct {
  const void* q_codes;            /* uint8 E4M3 [num_tokens, h_idx, 128], 16-byte aligned */
  const float* q_scales;          /* fp32 [num_tokens, h_idx] */
  const float* weights;           /* fp32 [num_tokens, h_idx] */
  int num_tokens, h_idx;          /* h_idx a multiple of 8, at most 256 */
  const int32_t* row_offsets;     /* int32 [batch + 1], non-decreasing, row_offsets[batch] = num_tokens */
  int batch;
  int max_new_tokens;             /* >= every element's row count; max_new_tokens * h_idx <= 256 */
  const void* k_codes;            /* uint8 E4M3 [num_pages, 64, 128], 16-byte aligned */
  const float* k_scales;          /* fp32 [num_pages, 64] */
  int num_pages, page_size;       /* page_size must be 64 */
  const int32_t* block_table;     /* int32 [batch, block_table_stride] */
  int block_table_stride;
  const int32_t* cache_seqlens;   /* int32 [batch], each <= block_table_stride * 64 */
  int relu;
  int topk;                       /* 1 .. 16384 */
  void* workspace;                /* >= mla_index_topk_workspace_size() bytes (fp32 scores) */
  size_t workspace_bytes;
  int32_t* indices;               /* out: int32 [num_tokens, topk] */
} mla_index_topk_args;

/* Scratch bytes for mla_index_topk: num_tokens x block_table_stride x 64 fp32 scores. */
mla_status mla_index_topk_workspace_size(int num_tokens, int block_table_stride, size_t* bytes);

/* Asynchronous on `stream`; device pointers owned by the caller.  Host-side
 * argument errors return without launching.  On the device, a block-table
 * entry outside [0, num_pages) sets MLA_DEVICE_BAD_PAGE (its keys are not
 * selected) and an element with more than max_new_tokens rows sets
 * MLA_DEVICE_BAD_SCHEDULE (its rows get -1). */
mla_status mla_index_topk(const mla_index_topk_args* args, mla_stream_t stream);

/* Test hooks, process-wide, for the library's own tests; production callers
 * never need them.  num_parts > 0 makes every later schedule (metadata,
 * workspace and decode geometry) use that many parts instead of the count
 * the SM count gives, to exercise split-KV paths on small inputs; 0 restores
 * the default.  debug_stall != 0 makes the decode kernel's softmax role wait
 * on a barrier that nothing completes, so that its bounded wait runs out and
 * MLA_DEVICE_TIMEOUT is reported; 0 restores normal operation.  The pages
 * describe no such call.  Returns MLA_ERR_INVALID_ARG for num_parts < 0. */
mla_status mla_test_hooks(int num_parts, int debug_stall);

/* Synchronises `stream`, returns the device status bits accumulated since the
 * last call in *flags (0 = clean) and clears them.  Returns
 * MLA_ERR_DEVICE_TIMEOUT / MLA_ERR_DEVICE_BOUNDS when the matching bit is set. */
mla_status mla_get_device_status(mla_stream_t stream, uint32_t* flags);

/* Thread-local description of the last error returned on this thread
 * (empty string if none).  The pointer stays valid until the next call. */
const char* mla_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MLA_H_ */
