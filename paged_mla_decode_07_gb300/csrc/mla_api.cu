// libmla host side: argument validation, geometry, TMA tensor maps, launches,
// device status and error reporting for the C ABI declared in include/mla.h.
//
// Error convention: each entry point checks every argument it can on the
// host and returns a status code without launching anything on failure; the
// thread-local message names the offending argument (the validation style of
// the MAX kernel wrappers, max.nn.kernels module overview).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <string>

#include "mla_internal.h"

namespace mla {

size_t metadata_smem_bytes(int np, int num_parts);

namespace {

thread_local std::string g_error;

mla_status fail(mla_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_error = buf;
  return s;
}

mla_status ok() {
  g_error.clear();
  return MLA_OK;
}

mla_status cuda_fail(cudaError_t e, const char* what) {
  return fail(MLA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Device status word: one per device (a module global), its address fetched
// once per device.
__device__ uint32_t g_device_status;
constexpr int kMaxDevices = 64;
uint32_t* g_status_ptr[kMaxDevices];
int g_sm_count[kMaxDevices];
int g_pair_capacity[kMaxDevices];  // co-resident CTA pairs of the pair decode kernel
int g_cluster_capacity[kMaxDevices][4];  // clusters of 1, 2, 4, 8 CTAs resident at once
std::mutex g_mu;

mla_status device_info(uint32_t** status, int* sm_count, int* pair_capacity = nullptr,
                       const int** cluster_capacity = nullptr) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(MLA_ERR_UNSUPPORTED, "device ordinal %d too large", dev);
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_status_ptr[dev]) {
    void* ptr = nullptr;
    e = cudaGetSymbolAddress(&ptr, g_device_status);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(status)");
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(SM count)");
    g_status_ptr[dev] = static_cast<uint32_t*>(ptr);
    g_sm_count[dev] = sms;
    const int cap = pair_cluster_capacity();
    g_pair_capacity[dev] = (cap > 0 && cap < sms / 2) ? cap : sms / 2;
    g_cluster_capacity[dev][0] = sms;
    for (int i = 1; i < 4; ++i) g_cluster_capacity[dev][i] = window_cluster_capacity(1 << i);
  }
  if (status) *status = g_status_ptr[dev];
  if (sm_count) *sm_count = g_sm_count[dev];
  if (pair_capacity) *pair_capacity = g_pair_capacity[dev];
  if (cluster_capacity) *cluster_capacity = g_cluster_capacity[dev];
  return MLA_OK;
}

// The CTA-pair decode kernel for problems of more than 64 rows, dense over
// the bf16 cache or sparse over FP8 or bf16 rows (mla_decode_pair.cu).
constexpr bool kPairDecode = true;
// Sparse on CTA pairs.
constexpr bool kPairSparse = true;

// Test hooks (mla_test_hooks): a forced part count and a stalled softmax role.
std::atomic<int> g_test_num_parts{0};
std::atomic<int> g_test_debug_stall{0};

// Kernel mode of a decode: 0 dense over the bf16 cache, 1 sparse over the FP8
// cache, 2 dense over the FP8 cache, 3 sparse over bf16 rows.
int decode_mode(int topk, int is_fp8) { return topk > 0 ? (is_fp8 ? 1 : 3) : (is_fp8 ? 2 : 0); }

mla_status geometry(int batch, int h_q, int s_q, int topk, int is_fp8, Geometry* g) {
  if (batch < 1) return fail(MLA_ERR_INVALID_ARG, "batch must be >= 1 (got %d)", batch);
  if (s_q < 1) return fail(MLA_ERR_INVALID_ARG, "s_q must be >= 1 (got %d)", s_q);
  if (h_q < 1) return fail(MLA_ERR_INVALID_ARG, "h_q must be >= 1 (got %d)", h_q);
  if (topk < 0) return fail(MLA_ERR_INVALID_ARG, "topk must be >= 0 (got %d)", topk);
  const long long np = topk > 0 ? static_cast<long long>(batch) * s_q : batch;
  const long long rows = topk > 0 ? h_q : static_cast<long long>(s_q) * h_q;
  if (np > kMaxProblems)
    return fail(MLA_ERR_UNSUPPORTED, "%s = %lld exceeds the supported %d problems",
                topk > 0 ? "batch*s_q" : "batch", np, kMaxProblems);
  if (rows > 1024)
    return fail(MLA_ERR_UNSUPPORTED, "%s = %lld query rows per problem exceeds 1024",
                topk > 0 ? "h_q" : "s_q*h_q", rows);
  if (topk > (1 << 24)) return fail(MLA_ERR_UNSUPPORTED, "topk = %d too large", topk);
  if (is_fp8 != 0 && is_fp8 != 1) return fail(MLA_ERR_INVALID_ARG, "is_fp8 must be 0 or 1 (got %d)", is_fp8);
  int sms = 0, pairs = 0;
  mla_status st = device_info(nullptr, &sms, &pairs);
  if (st != MLA_OK) return st;
  g->num_problems = static_cast<int>(np);
  g->rows = static_cast<int>(rows);
  g->mode = decode_mode(topk, is_fp8);
  g->sm_count = sms;
  // problems of more than 64 rows, dense over the bf16 cache or sparse (FP8
  // or bf16 rows), run on CTA pairs (128 rows and 128-token tiles per pair);
  // everything else on single CTAs
  g->pair = (kPairDecode && (g->mode == 0 || (kPairSparse && (g->mode == 1 || g->mode == 3))) && g->rows > 64)
                ? 1
                : 0;
  g->rpc = g->pair ? 128 : rows_per_cta(g->rows);
  g->tile_tokens = g->pair ? 128 : kTileTokens;
  g->row_groups = (g->rows + g->rpc - 1) / g->rpc;
  // persistent grids: one CTA (or CTA pair) per SM (or per pair of SMs that
  // can hold one) for every row group of a part
  g->num_parts = (g->pair ? pairs : sms) / g->row_groups;
  const int forced = g_test_num_parts.load();
  if (forced > 0) g->num_parts = forced;
  if (g->num_parts < 1) g->num_parts = 1;
  // schedule costs in quarters of a 64-token bf16 tile: FP8 rows are
  // dequantised before their MMAs, so their tiles weigh more against the
  // fixed start-up of a segment
  g->tile_cost = (is_fp8 ? 6 : 4) * (g->tile_tokens / kTileTokens);
  g->overhead = 8;
  g->tag = g->rpc | (g->mode << 8) | ((g->tile_tokens / kTileTokens) << 12) | (g->pair << 15);
  return MLA_OK;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Partial-result slots: only split problems take slots, at most two per part
// (see the metadata kernel), independent of the number of problems.
int max_slots(const Geometry& g) {
  // also at most one piece per problem plus one per part boundary
  return g.num_problems + g.num_parts < 2 * g.num_parts ? g.num_problems + g.num_parts : 2 * g.num_parts;
}

void workspace_layout(const Geometry& g, size_t* o_bytes, size_t* lse_bytes) {
  const size_t slots = static_cast<size_t>(max_slots(g));
  *o_bytes = align256(slots * g.rows * kDv * sizeof(float));
  *lse_bytes = align256(slots * g.rows * sizeof(float));
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// cuTensorMapEncodeTiled(args...).  A driver call, it wants the context current
// that a runtime call would make current: in a host thread whose first CUDA
// call this is there is none yet, and the current device's becomes it.
template <class... Args>
mla_status encode_map(const char* what, Args... args) {
  auto fn = encode_fn();
  if (!fn) return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled entry point unavailable");
  CUresult r = fn(args...);
  int dev = 0;
  if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess)
    r = fn(args...);
  if (r != CUDA_SUCCESS) return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed with CUresult %d", what, (int)r);
  return MLA_OK;
}

// 576-wide bf16 rows viewed as [rows][9 chunks][64]: dim0 = 64 elements
// (128 B, the swizzle atom width), dim1 = chunk (stride 128 B), dim2 = row
// (stride 1152 B).  A box of {64, 1, box_rows} lands in shared memory as
// box_rows x 128 B with the 128-byte swizzle, the canonical K-major operand
// layout of the tcgen05 MMAs.
mla_status encode_rows_map(CUtensorMap* map, const void* base, long long nrows, int box_rows, const char* what) {
  cuuint64_t dims[3] = {64, 9, static_cast<cuuint64_t>(nrows)};
  cuuint64_t strides[2] = {128, static_cast<cuuint64_t>(kDqk * 2)};
  cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode_map(what, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// The same 576-wide bf16 rows viewed chunk-major: dim0 = 64 elements of a
// chunk, dim1 = row (stride 1152 B), dim2 = chunk (stride 128 B).  A box of
// {64, 64, n} copies n chunks of 64 consecutive rows in one instruction and
// lands as n x [64 rows][128 B] with the 128-byte swizzle: n consecutive
// K-major operand tiles of the tcgen05 MMAs.
mla_status encode_chunk_major_map(CUtensorMap* map, const void* base, long long nrows, int box_chunks,
                                  const char* what) {
  cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(nrows), 9};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(kDqk * 2), 128};
  cuuint32_t box[3] = {64, 64, static_cast<cuuint32_t>(box_chunks)};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode_map(what, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// Cache rows as raw bytes, [rows][row_bytes] (row = page * 64 + slot, or the
// row of an unpaged KV): FP8 rows (656 bytes) or bf16 rows (1152 bytes).  A
// box is 128 bytes of box_rows rows: one row for the sparse row gathers (as
// row gathers require), 32 consecutive rows of a page for dense decode over
// the FP8 cache; no swizzle: the rows land as plain 128-byte rows.
mla_status encode_byte_rows_map(CUtensorMap* map, const void* base, long long nrows, int row_bytes, int box_rows) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(nrows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
  cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return encode_map("kv rows", map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
                    estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// E4M3 rows of 128 bytes, [rows][128], 128-byte swizzle: a box of box_rows
// rows lands as the canonical K-major operand of a kind::f8f6f4 MMA.
mla_status encode_e4m3_rows_map(CUtensorMap* map, const void* base, long long nrows, int box_rows, const char* what) {
  cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(nrows)};
  cuuint64_t strides[1] = {128};
  cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return encode_map(what, map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

uint64_t watchdog_ns() {
  const char* s = getenv("MLA_WATCHDOG_NS");
  if (s) {
    unsigned long long v = strtoull(s, nullptr, 10);
    if (v > 0) return v;
  }
  return 2000000000ull;  // 2 s: far above any legitimate wait, short enough to unwind quickly
}

}  // namespace

void set_error_message(const std::string& msg) { g_error = msg; }

}  // namespace mla

using namespace mla;

// Sparse prefill runs the decode pipeline (schedule, attention, combine) on
// chunks of at most kMaxProblems query tokens; the workspace holds one
// chunk's schedule, slot prefix sums and split-KV partials.
namespace {
struct PrefillLayout {
  size_t sched, num_splits, o_accum, lse_accum, total;
};
mla_status prefill_layout(int s_q, int h_q, int topk, Geometry* g, PrefillLayout* L) {
  const int chunk = s_q < kMaxProblems ? s_q : kMaxProblems;
  mla_status st = geometry(1, h_q, chunk, topk, 0, g);
  if (st != MLA_OK) return st;
  size_t ob, lb;
  workspace_layout(*g, &ob, &lb);
  L->sched = 0;
  L->num_splits = align256(static_cast<size_t>(g->num_parts) * kSchedInts * sizeof(int32_t));
  L->o_accum = L->num_splits + align256(static_cast<size_t>(chunk + 1) * sizeof(int32_t));
  L->lse_accum = L->o_accum + ob;
  L->total = L->lse_accum + lb;
  return MLA_OK;
}

// The register-level kernel (mla_decode_rows.cu) takes 16 query rows per CTA and
// reads the keys again for every 16: it runs windowed decode at up to 16 rows,
// and at more where all groups together have few pages for each SM to read.
// Measured (us, against the tcgen05 kernels): bf16, 128 elements x 16 rows x 4160
// keys 110.1 / 112.0; 4 x 16 x 512 keys 12.8 / 17.2; 32 rows, 4 x 512 keys 12.9 /
// 20.5, 30 x 512 (3.9 pages an SM) 18.5 / 24.7, 30 x 2048 (13.4) 39.0 / 35.1; 64
// rows, 16 x 512 (4.2) 17.8 / 24.0, 30 x 512 (7.9) 28.0 / 24.7.  FP8, 128 x 16 x
// 4160 keys 138 / 175; 64 rows, 16 x 512 19.5 / 24.0, 30 x 512 31.5 / 25.4.
constexpr int kRowsKernelRows = 16, kRowsKernelPages = 5;
bool rows_kernel(const Geometry& g, long long pages) {
  return g.rows <= kRowsKernelRows ||
         pages * g.num_problems * ((g.rows + 15) / 16) <= static_cast<long long>(kRowsKernelPages) * g.sm_count;
}
void rows_geometry(Geometry* g) {
  g->rpc = 16;
  g->row_groups = (g->rows + 15) / 16;
  g->pair = 0;
  g->mode = 7;
  g->tile_tokens = kTileTokens;
  g->tile_cost = 4;
  g->overhead = 4;  // a segment's start is about a page (16 rows, 64 elements: 61.1 us against 63.2 at 8)
  const int forced = g_test_num_parts.load();
  g->num_parts = forced > 0 ? forced : g->sm_count / g->row_groups;
  if (g->num_parts < 1) g->num_parts = 1;
}

// CTAs of the largest clusters, one for each row group of each problem, that
// have a page each and are resident at once; 0: none.
int largest_cluster(const Geometry& g, long long pages, const int* capacity) {
  if (g.pair || g_test_num_parts.load() > 0) return 0;
  const long long units = static_cast<long long>(g.num_problems) * g.row_groups;
  for (int i = 3; i >= 0; --i)
    if (units <= capacity[i] && (1 << i) <= pages) return 1 << i;
  return 0;
}

// CTAs of the cluster that each problem of a windowed call is given on the
// single-CTA kernels (mla_cluster.cuh), or 0 for a schedule over all SMs with a
// merge kernel behind it.  A cluster is taken when all of them are resident at
// once and the longest problem's share is at most three pages more than an even
// share of all pages: about what a schedule costs, its segments that start and
// end inside a problem, and the merge.  Measured (us, cluster against schedule,
// replayed, pages not in L2): the register-level kernel, 16 rows, bf16, windows
// of 512: 4 elements 11.9 / 13.8, 60 18.9 / 23.6, 150 29.6 / 35.3; of 2048: 34
// 26.3 / 29.4, but 16 elements 24.4 / 22.5 and 100 69.8 / 58.8; FP8, windows of
// 128: 4 10.3 / 12.8, 60 14.2 / 19.4, 128 20.4 / 25.5; of 1024: 100 53.3 / 46.9.  64
// rows on the tcgen05 kernels, windows of 512: 60 elements bf16 29.8 / 38.1, FP8
// 31.8 / 40.6.  Over 330 such calls (16 to 64 rows, 1 to 150 elements, windows of
// 128 to 4096) the side taken is within 5 % of the better one in all but 15; worst
// 19 % (4 x 16 rows x 2048 keys of bf16: schedule 20.7, cluster 17.3) and 16 % the
// other way (16 x 64 rows x 1024 keys of FP8: cluster 30.6, schedule 26.2).
int window_cluster(const Geometry& g, long long pages, const int* capacity) {
  const int n = largest_cluster(g, pages, capacity);
  const long long units = static_cast<long long>(g.num_problems) * g.row_groups;
  return pages * g.sm_count <= (pages * units + 3ll * g.sm_count) * n ? n : 0;
}

// Pages of all problems of a schedule that a call may have: the sums of a
// schedule made in the decode kernel have 31 bits for them.
constexpr long long kMaxTilesTotal = 1ll << 28;

// Windowed decode: spans of the problems and split-KV partials.  `pages`: the
// longest a window of the call can be, the lengths being on the device (the
// layout is largest where that is too long for the register-level kernel).
struct WindowLayout {
  size_t o_accum, lse_accum, total;  // (the spans come first)
};
mla_status window_layout(int batch, int h_q, int s_q, int is_fp8, long long pages, Geometry* g, WindowLayout* L) {
  mla_status st = geometry(batch, h_q, s_q, 0, is_fp8, g);
  if (st != MLA_OK) return st;
  g->mode = is_fp8 ? 5 : 4;
  // a segment on a CTA pair costs about four of its tiles to start and to end
  // (64 elements x 128 rows, 33 pages: 70.7 us against 73.0 at one and a half)
  if (g->pair) g->overhead = 32;
  if (rows_kernel(*g, pages)) rows_geometry(g);
  // two slots per part: the problems it starts and ends inside of
  const size_t slots = 2 * static_cast<size_t>(g->num_parts);
  L->o_accum = align256(static_cast<size_t>(g->num_problems) * 2 * sizeof(int32_t));
  L->lse_accum = L->o_accum + align256(slots * g->rows * kDv * sizeof(float));
  L->total = L->lse_accum + align256(slots * g->rows * sizeof(float));
  return MLA_OK;
}

// A small shared-prefix call runs as windowed ones do, each element over the
// prefix and its own keys on clusters of the register-level kernel: the prefix
// is then read for every 16 query rows, from L2.  Taken where a CTA has at most
// 8 (FP8: 14) pages.  Measured (us, against blocks of 128 rows): bf16, 16 rows,
// 6 elements behind 2000 keys (4.5 pages a CTA) 18.5 / 23.1, 32 (9) 26.7 / 29.5, 16
// (9) 26.0 / 24.7, 60 (18) 42.4 / 33.6; 128 rows, 4 behind 300 14.4 / 20.5; FP8,
// 16 rows, 6 behind 2000 20.3 / 34.8, behind 8000 (16) 46.5 / 48.7, 60 behind 2000
// (18) 50.7 / 43.3.
constexpr int kPrefixPagesEach = 8, kPrefixPagesEachFp8 = 14;

// Shared-prefix decode, on CTA pairs over blocks of 128 query rows (`pre`).
// bf16 rows: the prefix and the own keys in one.  FP8 rows: the prefix alone,
// as bf16 rows with a table of its pages; the own keys in a kernel of their
// own (`own`).
struct PrefixLayout {
  Geometry pre, own;
  int prefix_slots, own_slots;
  size_t spans, own_spans, o, lse, own_o, own_lse, table, rows, total;
};
mla_status prefix_layout(int batch, int h_q, int s_q, int prefix_pages, int is_fp8, PrefixLayout* L) {
  memset(L, 0, sizeof *L);
  mla_status st = geometry(batch, h_q, s_q, 0, is_fp8, &L->own);
  if (st != MLA_OK) return st;
  int pairs = 0;
  st = device_info(nullptr, nullptr, &pairs);
  if (st != MLA_OK) return st;
  const long long rows = static_cast<long long>(batch) * L->own.rows;
  if (is_fp8 && L->own.rows <= kRowsKernelRows) {
    rows_geometry(&L->own);
  } else if (is_fp8) {
    // the windowed mode with sinks that are every key
    L->own.mode = 5;
  }
  const long long np = (rows + 127) / 128;
  if (np > kMaxProblems)
    return fail(MLA_ERR_UNSUPPORTED, "batch*s_q*h_q = %lld query rows make %lld problems, more than the supported %d",
                rows, np, kMaxProblems);
  if (np * prefix_pages > kMaxTilesTotal)
    return fail(MLA_ERR_UNSUPPORTED, "batch*s_q*h_q = %lld query rows over a prefix table of %d entries", rows,
                prefix_pages);
  Geometry& g = L->pre;
  g = L->own;
  g.num_problems = static_cast<int>(np);
  g.rows = 128;
  g.rpc = 128;
  g.row_groups = 1;
  g.pair = 1;
  g.mode = 6;
  g.tile_tokens = 128;
  g.tile_cost = 8;
  // as for windows (64 x 128 rows behind 1000 keys: 50.9 us at two tiles, 48.5 at
  // four, 48.2 at five and a half; 8192 keys: 140.8, 140.8, 142.5)
  g.overhead = 32;
  const int forced = g_test_num_parts.load();
  g.num_parts = forced > 0 ? forced : (pairs > 0 ? pairs : 1);
  // FP8: every piece takes a slot, two per part and one per problem held whole
  L->prefix_slots = 2 * g.num_parts + (is_fp8 ? static_cast<int>(np) : 0);
  L->own_slots = is_fp8 ? 2 * L->own.num_parts + batch : 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  L->spans = take(static_cast<size_t>(np) * 8);
  L->own_spans = take(is_fp8 ? static_cast<size_t>(batch) * 8 : 0);
  L->o = take(static_cast<size_t>(L->prefix_slots) * 128 * kDv * 4);
  L->lse = take(static_cast<size_t>(L->prefix_slots) * 128 * 4);
  L->own_o = take(static_cast<size_t>(L->own_slots) * L->own.rows * kDv * 4);
  L->own_lse = take(static_cast<size_t>(L->own_slots) * L->own.rows * 4);
  if (is_fp8) {
    L->table = take(static_cast<size_t>(prefix_pages) * 4);
    L->rows = take(static_cast<size_t>(prefix_pages) * kPageSize * kDqk * 2);
  }
  L->total = at;
  return MLA_OK;
}

// Checks that every dense decode call over a paged cache shares.
mla_status check_paged(int batch, const void* q, const void* kvcache, const int32_t* block_table, const int32_t* cache_seqlens,
                       const void* out, const float* lse, int num_pages, int page_size, int stride, float sm_scale,
                       int is_fp8, const float* kv_scales) {
  if (!q) return fail(MLA_ERR_INVALID_ARG, "q is NULL");
  if (!kvcache) return fail(MLA_ERR_INVALID_ARG, "kvcache is NULL");
  if (!block_table) return fail(MLA_ERR_INVALID_ARG, "block_table is NULL");
  if (!cache_seqlens) return fail(MLA_ERR_INVALID_ARG, "cache_seqlens is NULL");
  if (!out) return fail(MLA_ERR_INVALID_ARG, "out is NULL");
  if (!lse) return fail(MLA_ERR_INVALID_ARG, "lse is NULL");
  if (page_size != kPageSize) return fail(MLA_ERR_UNSUPPORTED, "page_size must be %d (got %d)", kPageSize, page_size);
  if (num_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages must be >= 1 (got %d)", num_pages);
  if (num_pages > kMaxPages) return fail(MLA_ERR_UNSUPPORTED, "num_pages = %d exceeds 2^31 tokens", num_pages);
  if (stride < 1) return fail(MLA_ERR_INVALID_ARG, "block_table_stride must be >= 1 (got %d)", stride);
  if (static_cast<long long>(batch) * stride > kMaxTilesTotal)
    return fail(MLA_ERR_UNSUPPORTED, "a block table of %d x %d entries", batch, stride);
  if (!std::isfinite(sm_scale)) return fail(MLA_ERR_INVALID_ARG, "sm_scale is not finite");
  if (is_fp8 != 0 && is_fp8 != 1) return fail(MLA_ERR_INVALID_ARG, "is_fp8 must be 0 or 1 (got %d)", is_fp8);
  if (kv_scales && !is_fp8) return fail(MLA_ERR_INVALID_ARG, "kv_scales given with a bf16 cache (is_fp8 = 0)");
  if (!aligned(q, 16)) return fail(MLA_ERR_INVALID_ARG, "q is not 16-byte aligned");
  if (!aligned(kvcache, 16)) return fail(MLA_ERR_INVALID_ARG, "kvcache is not 16-byte aligned");
  if (!aligned(out, 16)) return fail(MLA_ERR_INVALID_ARG, "out is not 16-byte aligned");
  if (!aligned(lse, 4)) return fail(MLA_ERR_INVALID_ARG, "lse is not 4-byte aligned");
  if (!aligned(block_table, 4)) return fail(MLA_ERR_INVALID_ARG, "block_table is not 4-byte aligned");
  if (!aligned(cache_seqlens, 4)) return fail(MLA_ERR_INVALID_ARG, "cache_seqlens is not 4-byte aligned");
  if (!aligned(kv_scales, 4)) return fail(MLA_ERR_INVALID_ARG, "kv_scales is not 4-byte aligned");
  return MLA_OK;
}
mla_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (!workspace) return fail(MLA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
  if (bytes < need) return fail(MLA_ERR_WORKSPACE, "workspace_bytes = %zu < %zu needed", bytes, need);
  if (!aligned(workspace, 256)) return fail(MLA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  return MLA_OK;
}
// Tensor maps of the pair kernel over bf16 rows.
mla_status encode_pair_maps(const void* q, long long q_rows, const void* kv, long long kv_rows, CUtensorMap* tm_q,
                            CUtensorMap* tm_ks, CUtensorMap* tm_kv) {
  mla_status st = encode_chunk_major_map(tm_q, q, q_rows, kNumChunks, "q");
  if (st == MLA_OK) st = encode_chunk_major_map(tm_ks, kv, kv_rows, 3, "kvcache");
  if (st == MLA_OK) st = encode_chunk_major_map(tm_kv, kv, kv_rows, 2, "kvcache");
  return st;
}
}  // namespace

extern "C" {

int mla_abi_version(void) { return MLA_ABI_VERSION; }

const char* mla_last_error(void) { return g_error.c_str(); }

mla_status mla_test_hooks(int num_parts, int debug_stall) {
  if (num_parts < 0) return fail(MLA_ERR_INVALID_ARG, "num_parts must be >= 0 (got %d)", num_parts);
  g_test_num_parts.store(num_parts);
  g_test_debug_stall.store(debug_stall != 0 ? 1 : 0);
  return ok();
}

mla_status mla_metadata_size(int batch, int h_q, int s_q, int topk, int is_fp8, int* sched_elems,
                             int* num_splits_elems) {
  if (!sched_elems) return fail(MLA_ERR_INVALID_ARG, "sched_elems is NULL");
  if (!num_splits_elems) return fail(MLA_ERR_INVALID_ARG, "num_splits_elems is NULL");
  Geometry g{};
  mla_status st = geometry(batch, h_q, s_q, topk, is_fp8, &g);
  if (st != MLA_OK) return st;
  *sched_elems = g.num_parts * kSchedInts;
  *num_splits_elems = g.num_problems + 1;
  return ok();
}

mla_status mla_workspace_size(int batch, int h_q, int s_q, int topk, int is_fp8, size_t* bytes) {
  if (!bytes) return fail(MLA_ERR_INVALID_ARG, "bytes is NULL");
  Geometry g{};
  mla_status st = geometry(batch, h_q, s_q, topk, is_fp8, &g);
  if (st != MLA_OK) return st;
  size_t ob, lb;
  workspace_layout(g, &ob, &lb);
  *bytes = ob + lb;
  return ok();
}

mla_status mla_get_metadata(const int32_t* cache_seqlens, int batch, int h_q, int s_q, int topk, int is_fp8,
                            int32_t* sched, int32_t* num_splits, mla_stream_t stream) {
  if (!cache_seqlens) return fail(MLA_ERR_INVALID_ARG, "cache_seqlens is NULL");
  if (!sched) return fail(MLA_ERR_INVALID_ARG, "sched is NULL");
  if (!num_splits) return fail(MLA_ERR_INVALID_ARG, "num_splits is NULL");
  Geometry g{};
  mla_status st = geometry(batch, h_q, s_q, topk, is_fp8, &g);
  if (st != MLA_OK) return st;
  cudaError_t e = launch_metadata(cache_seqlens, s_q, topk, g, sched, num_splits,
                                  reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "metadata kernel launch");
  return ok();
}

mla_status mla_decode(const mla_decode_args* a, mla_stream_t stream) {
  if (!a) return fail(MLA_ERR_INVALID_ARG, "args is NULL");
  const bool sparse = a->topk > 0;
  if (a->topk < 0) return fail(MLA_ERR_INVALID_ARG, "topk must be >= 0 (got %d)", a->topk);
  if (!a->q) return fail(MLA_ERR_INVALID_ARG, "q is NULL");
  if (!a->kvcache) return fail(MLA_ERR_INVALID_ARG, "kvcache is NULL");
  if (!a->block_table) return fail(MLA_ERR_INVALID_ARG, "block_table is NULL");
  if (!a->cache_seqlens) return fail(MLA_ERR_INVALID_ARG, "cache_seqlens is NULL");
  if (!a->sched) return fail(MLA_ERR_INVALID_ARG, "sched is NULL");
  if (!a->num_splits) return fail(MLA_ERR_INVALID_ARG, "num_splits is NULL");
  if (!a->out) return fail(MLA_ERR_INVALID_ARG, "out is NULL");
  if (!a->lse) return fail(MLA_ERR_INVALID_ARG, "lse is NULL");
  if (sparse && !a->indices) return fail(MLA_ERR_INVALID_ARG, "indices is NULL with topk = %d", a->topk);
  if (!sparse && a->indices) return fail(MLA_ERR_INVALID_ARG, "indices given with topk = 0");
  if (a->page_size != kPageSize)
    return fail(MLA_ERR_UNSUPPORTED, "page_size must be %d (got %d)", kPageSize, a->page_size);
  if (a->num_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages must be >= 1 (got %d)", a->num_pages);
  if (static_cast<long long>(a->num_pages) * kPageSize > (1ll << 31) - 1)
    return fail(MLA_ERR_UNSUPPORTED, "num_pages = %d exceeds 2^31 tokens", a->num_pages);
  if (a->block_table_stride < 1)
    return fail(MLA_ERR_INVALID_ARG, "block_table_stride must be >= 1 (got %d)", a->block_table_stride);
  if (a->is_causal && sparse) return fail(MLA_ERR_UNSUPPORTED, "is_causal applies to dense mode only");
  if (a->kv_scales && !a->is_fp8) return fail(MLA_ERR_INVALID_ARG, "kv_scales given with a bf16 cache (is_fp8 = 0)");
  if (a->topk_lengths && !sparse) return fail(MLA_ERR_INVALID_ARG, "topk_lengths given with topk = 0");
  if (a->kv_scales && !aligned(a->kv_scales, 4)) return fail(MLA_ERR_INVALID_ARG, "kv_scales is not 4-byte aligned");
  if (!std::isfinite(a->sm_scale)) return fail(MLA_ERR_INVALID_ARG, "sm_scale is not finite");
  if (!aligned(a->q, 16)) return fail(MLA_ERR_INVALID_ARG, "q is not 16-byte aligned");
  if (!aligned(a->kvcache, 16)) return fail(MLA_ERR_INVALID_ARG, "kvcache is not 16-byte aligned");
  if (!aligned(a->out, 16)) return fail(MLA_ERR_INVALID_ARG, "out is not 16-byte aligned");
  if (!aligned(a->lse, 4)) return fail(MLA_ERR_INVALID_ARG, "lse is not 4-byte aligned");
  if (!aligned(a->block_table, 4)) return fail(MLA_ERR_INVALID_ARG, "block_table is not 4-byte aligned");

  if (a->is_fp8 != 0 && a->is_fp8 != 1) return fail(MLA_ERR_INVALID_ARG, "is_fp8 must be 0 or 1 (got %d)", a->is_fp8);
  Geometry g{};
  mla_status st = geometry(a->batch, a->h_q, a->s_q, a->topk, a->is_fp8, &g);
  if (st != MLA_OK) return st;
  size_t ob, lb;
  workspace_layout(g, &ob, &lb);
  if (!a->workspace) return fail(MLA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", ob + lb);
  if (a->workspace_bytes < ob + lb)
    return fail(MLA_ERR_WORKSPACE, "workspace_bytes = %zu < %zu needed", a->workspace_bytes, ob + lb);
  if (!aligned(a->workspace, 256)) return fail(MLA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");

  uint32_t* status = nullptr;
  st = device_info(&status, nullptr);
  if (st != MLA_OK) return st;

  CUtensorMap tm_q, tm_kv, tm_kv2;
  const long long qrows = static_cast<long long>(a->batch) * a->s_q * a->h_q;
  const long long cache_rows = static_cast<long long>(a->num_pages) * kPageSize;
  if (g.pair) {
    // chunk-major boxes: Q of a CTA in one copy; dense: a page's score operand
    // in three copies of three chunks, its value shares in copies of two
    // chunks.  Sparse: the rows are copied by the gather warps with cp.async
    // and the two cache maps go unused.
    st = encode_chunk_major_map(&tm_q, a->q, qrows, kNumChunks, "q");
    if (st == MLA_OK && g.mode == 0) st = encode_chunk_major_map(&tm_kv, a->kvcache, cache_rows, 3, "kvcache");
    if (st == MLA_OK && g.mode == 0) st = encode_chunk_major_map(&tm_kv2, a->kvcache, cache_rows, 2, "kvcache");
    if (st != MLA_OK) return st;
    if (g.mode == 1 || g.mode == 3) tm_kv = tm_kv2 = tm_q;
  } else {
    st = encode_rows_map(&tm_q, a->q, qrows, g.rpc, "q");
  }
  if (st != MLA_OK) return st;
  const int mode = g.mode;
  if (g.pair)
    ;  // maps encoded above
  else if (mode == 0)
    st = encode_rows_map(&tm_kv, a->kvcache, cache_rows, kPageSize, "kvcache");
  else if (mode == 3)
    st = encode_byte_rows_map(&tm_kv, a->kvcache, cache_rows, 2 * kDqk, 1);
  else
    st = encode_byte_rows_map(&tm_kv, a->kvcache, cache_rows, a->kv_scales ? 640 : kFp8RowBytes, mode == 1 ? 1 : 32);
  if (st != MLA_OK) return st;

  DecodeParams p;
  memset(&p, 0, sizeof p);
  p.block_table = a->block_table;
  p.cache_seqlens = a->cache_seqlens;
  p.indices = a->indices;
  p.sched = a->sched;
  p.num_splits = a->num_splits;
  p.kv_fp8 = static_cast<const uint8_t*>(a->kvcache);
  p.out = a->out;
  p.lse = a->lse;
  p.o_accum = static_cast<float*>(a->workspace);
  p.lse_accum = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + ob);
  p.status = status;
  p.timeout_ns = watchdog_ns();
  p.batch = a->batch;
  p.s_q = a->s_q;
  p.h_q = a->h_q;
  p.topk = a->topk;
  p.num_pages = a->num_pages;
  p.block_table_stride = a->block_table_stride;
  p.num_problems = g.num_problems;
  p.rows = g.rows;
  p.row_groups = g.row_groups;
  p.num_parts = g.num_parts;
  p.max_slots = max_slots(g);
  p.is_causal = a->is_causal ? 1 : 0;
  p.evict_first = (g.row_groups == 1 && !g.pair) ? 1 : 0;
  p.sched_tag = g.tag;
  p.debug_stall = g_test_debug_stall.load();
  p.scale_log2 = a->sm_scale * 1.4426950408889634f;
  p.kv_scales = a->kv_scales;
  p.topk_lengths = a->topk_lengths;
  p.fp8_rope_off = mode == 3 ? 2 * kDv : (a->kv_scales ? kDv : kFp8RopeOffset);
  p.rows16 = mode == 3 ? 1 : 0;

  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = g.pair ? launch_decode_pair(tm_q, tm_kv, tm_kv2, p, g.mode == 1 || g.mode == 3, s)
                         : launch_decode(tm_q, tm_kv, p, g.rpc, mode, s);
  if (e != cudaSuccess) return cuda_fail(e, "decode kernel launch");

  CombineParams cp;
  cp.num_splits = a->num_splits;
  cp.cache_seqlens = a->cache_seqlens;
  cp.s_q = a->s_q;
  cp.topk = a->topk;
  cp.o_accum = p.o_accum;
  cp.lse_accum = p.lse_accum;
  cp.out = a->out;
  cp.lse = a->lse;
  cp.num_problems = g.num_problems;
  cp.rows = g.rows;
  cp.max_slots = p.max_slots;
  cp.status = status;
  e = launch_combine(cp, s, true);
  if (e != cudaSuccess) return cuda_fail(e, "combine kernel launch");
  return ok();
}

mla_status mla_fp8_cache_store(const void* x, int num_tokens, const int32_t* input_row_offsets,
                               const int32_t* cache_lengths, int batch, const int32_t* block_table,
                               int block_table_stride, void* kvcache, int num_pages, int page_size,
                               mla_stream_t stream) {
  if (batch < 1) return fail(MLA_ERR_INVALID_ARG, "batch = %d must be >= 1", batch);
  if (num_tokens < 0) return fail(MLA_ERR_INVALID_ARG, "num_tokens = %d must be >= 0", num_tokens);
  if (page_size != kPageSize) return fail(MLA_ERR_UNSUPPORTED, "page_size must be 64 (got %d)", page_size);
  if (num_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages = %d must be >= 1", num_pages);
  if (block_table_stride < 1)
    return fail(MLA_ERR_INVALID_ARG, "block_table_stride = %d must be >= 1", block_table_stride);
  if (num_tokens > 0 && !x) return fail(MLA_ERR_INVALID_ARG, "x is NULL");
  if (!input_row_offsets) return fail(MLA_ERR_INVALID_ARG, "input_row_offsets is NULL");
  if (!cache_lengths) return fail(MLA_ERR_INVALID_ARG, "cache_lengths is NULL");
  if (!block_table) return fail(MLA_ERR_INVALID_ARG, "block_table is NULL");
  if (!kvcache) return fail(MLA_ERR_INVALID_ARG, "kvcache is NULL");
  if (x && !aligned(x, 16)) return fail(MLA_ERR_INVALID_ARG, "x is not 16-byte aligned");
  if (!aligned(kvcache, 16)) return fail(MLA_ERR_INVALID_ARG, "kvcache is not 16-byte aligned");
  uint32_t* status = nullptr;
  int sms = 0;
  mla_status st = device_info(&status, &sms);
  if (st != MLA_OK) return st;
  cudaError_t e = launch_fp8_cache_store(static_cast<const uint16_t*>(x), num_tokens, input_row_offsets,
                                         cache_lengths, batch, block_table, block_table_stride,
                                         static_cast<uint8_t*>(kvcache), num_pages, status, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "fp8 cache store launch");
  return ok();
}

mla_status mla_cache_store(const mla_cache_store_args* a, mla_stream_t stream) {
  if (!a) return fail(MLA_ERR_INVALID_ARG, "args is NULL");
  if (a->num_tokens < 0) return fail(MLA_ERR_INVALID_ARG, "num_tokens must be >= 0 (got %d)", a->num_tokens);
  if (a->page_size != kPageSize) return fail(MLA_ERR_UNSUPPORTED, "page_size must be 64 (got %d)", a->page_size);
  if (a->num_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages must be >= 1 (got %d)", a->num_pages);
  if (a->num_pages > kMaxPages) return fail(MLA_ERR_UNSUPPORTED, "num_pages = %d exceeds 2^31 tokens", a->num_pages);
  if (a->is_fp8 != 0 && a->is_fp8 != 1) return fail(MLA_ERR_INVALID_ARG, "is_fp8 must be 0 or 1 (got %d)", a->is_fp8);
  if (a->kv_scales && !a->is_fp8) return fail(MLA_ERR_INVALID_ARG, "kv_scales given with a bf16 cache (is_fp8 = 0)");
  if (!a->kvcache) return fail(MLA_ERR_INVALID_ARG, "kvcache is NULL");
  if (!aligned(a->kvcache, 16)) return fail(MLA_ERR_INVALID_ARG, "kvcache is not 16-byte aligned");
  if (a->kv_scales && !aligned(a->kv_scales, 4)) return fail(MLA_ERR_INVALID_ARG, "kv_scales is not 4-byte aligned");
  if (a->latent_stride < 0 || a->latent_stride % 8 != 0)
    return fail(MLA_ERR_INVALID_ARG, "latent_stride must be a multiple of 8 elements (got %lld)",
                static_cast<long long>(a->latent_stride));
  if (a->rope_stride < 0 || a->rope_stride % 8 != 0)
    return fail(MLA_ERR_INVALID_ARG, "rope_stride must be a multiple of 8 elements (got %lld)",
                static_cast<long long>(a->rope_stride));
  if (a->num_tokens == 0) return ok();
  if (!a->latent) return fail(MLA_ERR_INVALID_ARG, "latent is NULL");
  if (!a->rope) return fail(MLA_ERR_INVALID_ARG, "rope is NULL");
  if (!a->slot_map) return fail(MLA_ERR_INVALID_ARG, "slot_map is NULL");
  if (!aligned(a->latent, 16)) return fail(MLA_ERR_INVALID_ARG, "latent is not 16-byte aligned");
  if (!aligned(a->rope, 16)) return fail(MLA_ERR_INVALID_ARG, "rope is not 16-byte aligned");
  if (!aligned(a->slot_map, 4)) return fail(MLA_ERR_INVALID_ARG, "slot_map is not 4-byte aligned");
  uint32_t* status = nullptr;
  int sms = 0;
  mla_status st = device_info(&status, &sms);
  if (st != MLA_OK) return st;
  SlotStoreParams p;
  memset(&p, 0, sizeof p);
  p.latent = static_cast<const uint16_t*>(a->latent);
  p.rope = static_cast<const uint16_t*>(a->rope);
  p.slots = a->slot_map;
  p.kvcache = static_cast<uint8_t*>(a->kvcache);
  p.kv_scales = a->kv_scales;
  p.status = status;
  p.latent_stride = a->latent_stride;
  p.rope_stride = a->rope_stride;
  p.num_tokens = a->num_tokens;
  p.num_slots = a->num_pages * kPageSize;
  p.is_fp8 = a->is_fp8;
  cudaError_t e = launch_slot_store(p, sms, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cache store launch");
  return ok();
}

mla_status mla_assign_pages(const mla_assign_pages_args* a, mla_stream_t stream) {
  if (!a) return fail(MLA_ERR_INVALID_ARG, "args is NULL");
  if (a->batch < 1) return fail(MLA_ERR_INVALID_ARG, "batch must be >= 1 (got %d)", a->batch);
  if (a->batch > kMaxProblems)
    return fail(MLA_ERR_UNSUPPORTED, "batch = %d exceeds the supported %d requests", a->batch, kMaxProblems);
  if (a->num_free < 0) return fail(MLA_ERR_INVALID_ARG, "num_free must be >= 0 (got %d)", a->num_free);
  if (a->num_tokens < 0) return fail(MLA_ERR_INVALID_ARG, "num_tokens must be >= 0 (got %d)", a->num_tokens);
  if (a->num_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages must be >= 1 (got %d)", a->num_pages);
  if (a->num_pages > kMaxPages) return fail(MLA_ERR_UNSUPPORTED, "num_pages = %d exceeds 2^31 tokens", a->num_pages);
  if (a->block_table_stride < 1)
    return fail(MLA_ERR_INVALID_ARG, "block_table_stride must be >= 1 (got %d)", a->block_table_stride);
  struct Arr {
    const void* p;
    long long n;  // int32 entries
    const char* name;
  };
  const Arr in[4] = {{a->cache_lengths, a->batch, "cache_lengths"},
                     {a->new_tokens, a->batch, "new_tokens"},
                     {a->free_pages, a->num_free, "free_pages"},
                     {a->free_cursor, 1, "free_cursor"}};
  const Arr out[5] = {{a->block_table, static_cast<long long>(a->batch) * a->block_table_stride, "block_table"},
                      {a->cache_seqlens, a->batch, "cache_seqlens"},
                      {a->row_offsets, a->batch + 1ll, "row_offsets"},
                      {a->slot_map, a->num_tokens, "slot_map"},
                      {a->next_cursor, 1, "next_cursor"}};
  for (const Arr& x : in) {
    if (!x.p && x.n > 0) return fail(MLA_ERR_INVALID_ARG, "%s is NULL", x.name);
    if (!aligned(x.p, 4)) return fail(MLA_ERR_INVALID_ARG, "%s is not 4-byte aligned", x.name);
  }
  for (const Arr& x : out) {
    if (!x.p && x.n > 0) return fail(MLA_ERR_INVALID_ARG, "%s is NULL", x.name);
    if (!aligned(x.p, 4)) return fail(MLA_ERR_INVALID_ARG, "%s is not 4-byte aligned", x.name);
  }
  // outputs overlap nothing, except that the lengths and the cursor may be
  // updated in the very arrays they are read from
  auto overlap = [](const Arr& x, const Arr& y) {
    const uintptr_t xs = reinterpret_cast<uintptr_t>(x.p), ys = reinterpret_cast<uintptr_t>(y.p);
    return x.n > 0 && y.n > 0 && xs < ys + 4 * static_cast<uintptr_t>(y.n) && ys < xs + 4 * static_cast<uintptr_t>(x.n);
  };
  for (int i = 0; i < 5; ++i) {
    for (int k = 0; k < 4; ++k) {
      const bool same = (i == 1 && k == 0 && out[i].p == in[k].p) || (i == 4 && k == 3 && out[i].p == in[k].p);
      if (!same && overlap(out[i], in[k]))
        return fail(MLA_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, in[k].name);
    }
    for (int k = 0; k < i; ++k)
      if (overlap(out[i], out[k])) return fail(MLA_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[k].name);
  }
  uint32_t* status = nullptr;
  int sms = 0;
  mla_status st = device_info(&status, &sms);
  if (st != MLA_OK) return st;
  AssignPagesParams p;
  memset(&p, 0, sizeof p);
  p.cache_lengths = a->cache_lengths;
  p.new_tokens = a->new_tokens;
  p.free_pages = a->free_pages;
  p.free_cursor = a->free_cursor;
  p.block_table = a->block_table;
  p.cache_seqlens = a->cache_seqlens;
  p.row_offsets = a->row_offsets;
  p.slot_map = a->num_tokens > 0 ? a->slot_map : nullptr;
  p.next_cursor = a->next_cursor;
  p.status = status;
  p.batch = a->batch;
  p.num_free = a->num_free;
  p.block_table_stride = a->block_table_stride;
  p.num_pages = a->num_pages;
  p.num_tokens = a->num_tokens;
  const bool in_place = a->cache_seqlens == a->cache_lengths || a->next_cursor == a->free_cursor;
  cudaError_t e = launch_assign_pages(p, in_place, sms, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "page assignment launch");
  return ok();
}

mla_status mla_sparse_prefill_workspace_size(int s_q, int h_q, int topk, size_t* bytes) {
  if (!bytes) return fail(MLA_ERR_INVALID_ARG, "bytes is NULL");
  if (topk < 1) return fail(MLA_ERR_INVALID_ARG, "topk must be >= 1 (got %d)", topk);
  Geometry g{};
  PrefillLayout L{};
  mla_status st = prefill_layout(s_q, h_q, topk, &g, &L);
  if (st != MLA_OK) return st;
  *bytes = L.total;
  return ok();
}

mla_status mla_sparse_prefill(const mla_sparse_prefill_args* a, mla_stream_t stream) {
  if (!a) return fail(MLA_ERR_INVALID_ARG, "args is NULL");
  if (!a->q) return fail(MLA_ERR_INVALID_ARG, "q is NULL");
  if (!a->kv) return fail(MLA_ERR_INVALID_ARG, "kv is NULL");
  if (!a->indices) return fail(MLA_ERR_INVALID_ARG, "indices is NULL");
  if (!a->out) return fail(MLA_ERR_INVALID_ARG, "out is NULL");
  if (!a->lse) return fail(MLA_ERR_INVALID_ARG, "lse is NULL");
  if (a->s_q < 1) return fail(MLA_ERR_INVALID_ARG, "s_q must be >= 1 (got %d)", a->s_q);
  if (a->s_kv < 1) return fail(MLA_ERR_INVALID_ARG, "s_kv must be >= 1 (got %d)", a->s_kv);
  if (a->topk < 1) return fail(MLA_ERR_INVALID_ARG, "topk must be >= 1 (got %d)", a->topk);
  if (!std::isfinite(a->sm_scale)) return fail(MLA_ERR_INVALID_ARG, "sm_scale is not finite");
  if (!aligned(a->q, 16)) return fail(MLA_ERR_INVALID_ARG, "q is not 16-byte aligned");
  if (!aligned(a->kv, 16)) return fail(MLA_ERR_INVALID_ARG, "kv is not 16-byte aligned");
  if (!aligned(a->out, 16)) return fail(MLA_ERR_INVALID_ARG, "out is not 16-byte aligned");
  if (!aligned(a->lse, 4)) return fail(MLA_ERR_INVALID_ARG, "lse is not 4-byte aligned");
  if (!aligned(a->indices, 4)) return fail(MLA_ERR_INVALID_ARG, "indices is not 4-byte aligned");
  Geometry g{};
  PrefillLayout L{};
  mla_status st = prefill_layout(a->s_q, a->h_q, a->topk, &g, &L);
  if (st != MLA_OK) return st;
  if (!a->workspace) return fail(MLA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", L.total);
  if (a->workspace_bytes < L.total)
    return fail(MLA_ERR_WORKSPACE, "workspace_bytes = %zu < %zu needed", a->workspace_bytes, L.total);
  if (!aligned(a->workspace, 256)) return fail(MLA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  uint32_t* status = nullptr;
  st = device_info(&status, nullptr);
  if (st != MLA_OK) return st;

  char* ws = static_cast<char*>(a->workspace);
  int32_t* sched = reinterpret_cast<int32_t*>(ws + L.sched);
  int32_t* num_splits = reinterpret_cast<int32_t*>(ws + L.num_splits);
  CUtensorMap tm_kv;
  st = encode_byte_rows_map(&tm_kv, a->kv, a->s_kv, 2 * kDqk, 1);
  if (st != MLA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const uint64_t timeout = watchdog_ns();
  for (int c0 = 0; c0 < a->s_q; c0 += kMaxProblems) {
    const int chunk = a->s_q - c0 < kMaxProblems ? a->s_q - c0 : kMaxProblems;
    Geometry gc{};
    st = geometry(1, a->h_q, chunk, a->topk, 0, &gc);
    if (st != MLA_OK) return st;
    const char* q = static_cast<const char*>(a->q) + static_cast<size_t>(c0) * a->h_q * kDqk * 2;
    CUtensorMap tm_q;
    st = gc.pair ? encode_chunk_major_map(&tm_q, q, static_cast<long long>(chunk) * a->h_q, kNumChunks, "q")
                 : encode_rows_map(&tm_q, q, static_cast<long long>(chunk) * a->h_q, gc.rpc, "q");
    if (st != MLA_OK) return st;
    cudaError_t e = launch_metadata(nullptr, chunk, a->topk, gc, sched, num_splits, s);
    if (e != cudaSuccess) return cuda_fail(e, "metadata kernel launch");

    DecodeParams p;
    memset(&p, 0, sizeof p);
    p.indices = a->indices + static_cast<size_t>(c0) * a->topk;
    p.sched = sched;
    p.num_splits = num_splits;
    p.kv_fp8 = static_cast<const uint8_t*>(a->kv);
    p.out = static_cast<char*>(a->out) + static_cast<size_t>(c0) * a->h_q * kDv * 2;
    p.lse = a->lse + static_cast<size_t>(c0) * a->h_q;
    p.o_accum = reinterpret_cast<float*>(ws + L.o_accum);
    p.lse_accum = reinterpret_cast<float*>(ws + L.lse_accum);
    p.status = status;
    p.timeout_ns = timeout;
    p.batch = 1;
    p.s_q = chunk;
    p.h_q = a->h_q;
    p.topk = a->topk;
    p.num_pages = 1;
    p.block_table_stride = 1;
    p.num_problems = gc.num_problems;
    p.rows = gc.rows;
    p.row_groups = gc.row_groups;
    p.num_parts = gc.num_parts;
    p.max_slots = max_slots(gc);
    p.evict_first = (gc.row_groups == 1 && !gc.pair) ? 1 : 0;
    p.sched_tag = gc.tag;
    p.flat_rows = a->s_kv;
    p.scale_log2 = a->sm_scale * 1.4426950408889634f;
    p.fp8_rope_off = 2 * kDv;
    p.rows16 = 1;
    e = gc.pair ? launch_decode_pair(tm_q, tm_q, tm_q, p, true, s) : launch_decode(tm_q, tm_kv, p, gc.rpc, 3, s);
    if (e != cudaSuccess) return cuda_fail(e, "sparse prefill attention kernel launch");
    CombineParams cp;
    cp.num_splits = num_splits;
    cp.cache_seqlens = nullptr;
    cp.s_q = chunk;
    cp.topk = a->topk;
    cp.o_accum = p.o_accum;
    cp.lse_accum = p.lse_accum;
    cp.out = p.out;
    cp.lse = p.lse;
    cp.num_problems = gc.num_problems;
    cp.rows = gc.rows;
    cp.max_slots = p.max_slots;
    cp.status = status;
    e = launch_combine(cp, s, true);
    if (e != cudaSuccess) return cuda_fail(e, "combine kernel launch");
  }
  return ok();
}

mla_status mla_window_decode_workspace_size(int batch, int h_q, int s_q, int is_fp8, size_t* bytes) {
  if (!bytes) return fail(MLA_ERR_INVALID_ARG, "bytes is NULL");
  Geometry g{};
  WindowLayout L{};
  mla_status st = window_layout(batch, h_q, s_q, is_fp8, kMaxPages, &g, &L);
  if (st != MLA_OK) return st;
  *bytes = L.total;
  return ok();
}

mla_status mla_window_decode(const mla_window_decode_args* a, mla_stream_t stream) {
  if (!a) return fail(MLA_ERR_INVALID_ARG, "args is NULL");
  mla_status st = check_paged(a->batch, a->q, a->kvcache, a->block_table, a->cache_seqlens, a->out, a->lse, a->num_pages,
                              a->page_size, a->block_table_stride, a->sm_scale, a->is_fp8, a->kv_scales);
  if (st != MLA_OK) return st;
  if (a->window < 1) return fail(MLA_ERR_INVALID_ARG, "window must be >= 1 (got %d)", a->window);
  if (a->sinks < 0) return fail(MLA_ERR_INVALID_ARG, "sinks must be >= 0 (got %d)", a->sinks);
  Geometry g{};
  WindowLayout L{};
  const long long reach = std::min<long long>(a->window, kMaxWindow) + a->s_q + a->sinks;
  const long long pages = std::min<long long>(a->block_table_stride, reach / kPageSize + 3);
  st = window_layout(a->batch, a->h_q, a->s_q, a->is_fp8, pages, &g, &L);
  if (st != MLA_OK) return st;
  st = check_workspace(a->workspace, a->workspace_bytes, L.total);
  if (st != MLA_OK) return st;
  uint32_t* status = nullptr;
  const int* clusters = nullptr;
  st = device_info(&status, nullptr, nullptr, &clusters);
  if (st != MLA_OK) return st;

  CUtensorMap tm_q, tm_kv, tm_kv2;
  const long long qrows = static_cast<long long>(a->batch) * a->s_q * a->h_q;
  const long long cache_rows = static_cast<long long>(a->num_pages) * kPageSize;
  if (g.pair) {
    st = encode_pair_maps(a->q, qrows, a->kvcache, cache_rows, &tm_q, &tm_kv, &tm_kv2);
  } else if (g.mode == 7) {
    memset(&tm_kv, 0, sizeof tm_kv);
    if (!a->is_fp8) st = encode_rows_map(&tm_kv, a->kvcache, cache_rows, kPageSize / 2, "kvcache");
  } else {
    st = encode_rows_map(&tm_q, a->q, qrows, g.rpc, "q");
    if (st == MLA_OK)
      st = a->is_fp8 ? encode_byte_rows_map(&tm_kv, a->kvcache, cache_rows, a->kv_scales ? 640 : kFp8RowBytes, 32)
                     : encode_rows_map(&tm_kv, a->kvcache, cache_rows, kPageSize, "kvcache");
  }
  if (st != MLA_OK) return st;

  char* ws = static_cast<char*>(a->workspace);
  DecodeParams p;
  memset(&p, 0, sizeof p);
  p.block_table = a->block_table;
  p.cache_seqlens = a->cache_seqlens;
  p.spans = reinterpret_cast<int32_t*>(ws);
  p.tile_cost = g.tile_cost;
  p.overhead = g.overhead;
  p.kv_fp8 = static_cast<const uint8_t*>(a->kvcache);
  p.out = a->out;
  p.lse = a->lse;
  p.o_accum = reinterpret_cast<float*>(ws + L.o_accum);
  p.lse_accum = reinterpret_cast<float*>(ws + L.lse_accum);
  p.status = status;
  p.timeout_ns = watchdog_ns();
  p.batch = a->batch;
  p.s_q = a->s_q;
  p.h_q = a->h_q;
  p.num_pages = a->num_pages;
  p.block_table_stride = a->block_table_stride;
  p.num_problems = g.num_problems;
  p.rows = g.rows;
  p.row_groups = g.row_groups;
  p.num_parts = g.num_parts;
  p.max_slots = 2 * g.num_parts;
  p.is_causal = 1;  // a window ends at its query token
  p.window = a->window < kMaxWindow ? a->window : kMaxWindow;
  p.sinks = a->sinks;
  p.evict_first = (g.row_groups == 1 && !g.pair) ? 1 : 0;
  p.debug_stall = g_test_debug_stall.load();
  p.scale_log2 = a->sm_scale * 1.4426950408889634f;
  p.kv_scales = a->kv_scales;
  p.fp8_rope_off = a->kv_scales ? kDv : kFp8RopeOffset;

  p.cluster = window_cluster(g, pages, clusters);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  e = g.pair        ? launch_window_pair(tm_q, tm_kv, tm_kv2, p, s)
      : g.mode == 7 ? launch_decode_rows(tm_kv, a->q, p, a->is_fp8, s)
                    : launch_decode(tm_q, tm_kv, p, g.rpc, g.mode, s);
  if (e != cudaSuccess) return cuda_fail(e, "window decode kernel launch");
  if (p.cluster > 0) return ok();  // (the cluster has merged)
  MergeParams m;
  memset(&m, 0, sizeof m);
  m.own = MergeSide{p.spans, p.o_accum, p.lse_accum, -1};
  m.rows = g.rows;
  m.problems = a->batch;
  m.total_rows = static_cast<int>(qrows);
  m.out = a->out;
  m.lse = a->lse;
  e = launch_merge(m, s);
  if (e != cudaSuccess) return cuda_fail(e, "merge kernel launch");
  return ok();
}

mla_status mla_shared_prefix_decode_workspace_size(int batch, int h_q, int s_q, int prefix_table_len, int is_fp8,
                                                   size_t* bytes) {
  if (!bytes) return fail(MLA_ERR_INVALID_ARG, "bytes is NULL");
  if (prefix_table_len < 1)
    return fail(MLA_ERR_INVALID_ARG, "prefix_table_len must be >= 1 (got %d)", prefix_table_len);
  if (prefix_table_len > kMaxPages)
    return fail(MLA_ERR_UNSUPPORTED, "prefix_table_len = %d exceeds 2^31 tokens", prefix_table_len);
  PrefixLayout L;
  mla_status st = prefix_layout(batch, h_q, s_q, prefix_table_len, is_fp8, &L);
  if (st != MLA_OK) return st;
  *bytes = L.total;
  return ok();
}

mla_status mla_shared_prefix_decode(const mla_shared_prefix_decode_args* a, mla_stream_t stream) {
  if (!a) return fail(MLA_ERR_INVALID_ARG, "args is NULL");
  mla_status st = check_paged(a->batch, a->q, a->kvcache, a->block_table, a->cache_seqlens, a->out, a->lse, a->num_pages,
                              a->page_size, a->block_table_stride, a->sm_scale, a->is_fp8, a->kv_scales);
  if (st != MLA_OK) return st;
  if (!a->prefix_table) return fail(MLA_ERR_INVALID_ARG, "prefix_table is NULL");
  if (!a->prefix_length) return fail(MLA_ERR_INVALID_ARG, "prefix_length is NULL");
  if (!aligned(a->prefix_table, 4)) return fail(MLA_ERR_INVALID_ARG, "prefix_table is not 4-byte aligned");
  if (!aligned(a->prefix_length, 4)) return fail(MLA_ERR_INVALID_ARG, "prefix_length is not 4-byte aligned");
  size_t need = 0;
  st = mla_shared_prefix_decode_workspace_size(a->batch, a->h_q, a->s_q, a->prefix_table_len, a->is_fp8, &need);
  if (st != MLA_OK) return st;
  st = check_workspace(a->workspace, a->workspace_bytes, need);
  if (st != MLA_OK) return st;
  PrefixLayout L;
  st = prefix_layout(a->batch, a->h_q, a->s_q, a->prefix_table_len, a->is_fp8, &L);
  if (st != MLA_OK) return st;
  uint32_t* status = nullptr;
  int sms = 0;
  const int* clusters = nullptr;
  st = device_info(&status, &sms, nullptr, &clusters);
  if (st != MLA_OK) return st;

  char* ws = static_cast<char*>(a->workspace);
  const long long qrows = static_cast<long long>(a->batch) * L.own.rows;
  const long long cache_rows = static_cast<long long>(a->num_pages) * kPageSize;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const long long pages = static_cast<long long>(a->prefix_table_len) + a->block_table_stride;
  Geometry g = L.own;
  rows_geometry(&g);
  const int cluster = largest_cluster(g, pages, clusters);
  if (cluster > 0 && pages <= (a->is_fp8 ? kPrefixPagesEachFp8 : kPrefixPagesEach) * static_cast<long long>(cluster)) {
    CUtensorMap tm_kv;
    memset(&tm_kv, 0, sizeof tm_kv);
    if (!a->is_fp8) st = encode_rows_map(&tm_kv, a->kvcache, cache_rows, kPageSize / 2, "kvcache");
    if (st != MLA_OK) return st;
    DecodeParams p;
    memset(&p, 0, sizeof p);
    p.block_table = a->block_table;
    p.cache_seqlens = a->cache_seqlens;
    p.kv_fp8 = static_cast<const uint8_t*>(a->kvcache);
    p.out = a->out;
    p.lse = a->lse;
    p.status = status;
    p.timeout_ns = watchdog_ns();
    p.batch = a->batch;
    p.s_q = a->s_q;
    p.h_q = a->h_q;
    p.num_pages = a->num_pages;
    p.block_table_stride = a->block_table_stride;
    p.num_problems = g.num_problems;
    p.rows = g.rows;
    p.row_groups = g.row_groups;
    p.num_parts = g.num_parts;
    p.is_causal = a->is_causal ? 1 : 0;
    p.window = 1;
    p.sinks = 0x7fffffff;  // every own key
    p.cluster = cluster;
    p.debug_stall = g_test_debug_stall.load();
    p.scale_log2 = a->sm_scale * 1.4426950408889634f;
    p.kv_scales = a->kv_scales;
    p.prefix_table = a->prefix_table;
    p.prefix_len = a->prefix_length;
    p.prefix_pages = a->prefix_table_len;
    cudaError_t e = launch_decode_rows(tm_kv, a->q, p, a->is_fp8, s);
    if (e != cudaSuccess) return cuda_fail(e, "shared-prefix decode kernel launch");
    return ok();
  }
  CUtensorMap tm_q, tm_ks, tm_kv, tm_own_q, tm_own_kv;
  if (a->is_fp8) {
    st = encode_pair_maps(a->q, qrows, ws + L.rows, static_cast<long long>(a->prefix_table_len) * kPageSize, &tm_q,
                          &tm_ks, &tm_kv);
    const int row_bytes = a->kv_scales ? 640 : kFp8RowBytes;
    if (L.own.mode != 7) {
      if (st == MLA_OK) st = encode_rows_map(&tm_own_q, a->q, qrows, L.own.rpc, "q");
      if (st == MLA_OK) st = encode_byte_rows_map(&tm_own_kv, a->kvcache, cache_rows, row_bytes, 32);
    }
  } else {
    st = encode_pair_maps(a->q, qrows, a->kvcache, cache_rows, &tm_q, &tm_ks, &tm_kv);
  }
  if (st != MLA_OK) return st;

  cudaError_t e = cudaSuccess;
  DecodeParams p;
  memset(&p, 0, sizeof p);
  p.block_table = a->block_table;
  p.cache_seqlens = a->cache_seqlens;
  p.spans = reinterpret_cast<int32_t*>(ws + L.spans);
  p.tile_cost = L.pre.tile_cost;
  p.overhead = L.pre.overhead;
  p.o_accum = reinterpret_cast<float*>(ws + L.o);
  p.lse_accum = reinterpret_cast<float*>(ws + L.lse);
  p.out = a->out;
  p.lse = a->lse;
  p.status = status;
  p.timeout_ns = watchdog_ns();
  p.batch = a->batch;
  p.s_q = a->s_q;
  p.h_q = a->h_q;
  p.num_pages = a->is_fp8 ? a->prefix_table_len : a->num_pages;
  p.block_table_stride = a->block_table_stride;
  p.num_problems = L.pre.num_problems;
  p.rows = L.own.rows;
  p.row_groups = 1;
  p.num_parts = L.pre.num_parts;
  p.max_slots = L.prefix_slots;
  p.always_partial = a->is_fp8;
  p.is_causal = a->is_causal ? 1 : 0;
  p.debug_stall = g_test_debug_stall.load();
  p.scale_log2 = a->sm_scale * 1.4426950408889634f;
  p.prefix_table = a->is_fp8 ? reinterpret_cast<const int32_t*>(ws + L.table) : a->prefix_table;
  p.prefix_len = a->prefix_length;
  p.prefix_pages = a->prefix_table_len;
  p.total_rows = static_cast<int>(qrows);
  p.own_keys = !a->is_fp8;

  if (a->is_fp8) {
    e = launch_prefix_rows(static_cast<const uint8_t*>(a->kvcache), a->kv_scales, a->prefix_table, a->prefix_length,
                           a->prefix_table_len, a->num_pages, ws + L.rows, reinterpret_cast<int32_t*>(ws + L.table),
                           status, sms, s);
    if (e != cudaSuccess) return cuda_fail(e, "prefix rows kernel launch");
  }
  e = launch_prefix_pair(tm_q, tm_ks, tm_kv, p, s);
  if (e != cudaSuccess) return cuda_fail(e, "shared-prefix decode kernel launch");
  if (a->is_fp8) {
    DecodeParams o = p;
    o.spans = reinterpret_cast<int32_t*>(ws + L.own_spans);
    o.tile_cost = L.own.tile_cost;
    o.overhead = L.own.overhead;
    o.kv_fp8 = static_cast<const uint8_t*>(a->kvcache);
    o.o_accum = reinterpret_cast<float*>(ws + L.own_o);
    o.lse_accum = reinterpret_cast<float*>(ws + L.own_lse);
    o.num_pages = a->num_pages;
    o.num_problems = L.own.num_problems;
    o.row_groups = L.own.row_groups;
    o.num_parts = L.own.num_parts;
    o.max_slots = L.own_slots;
    o.prefix_len = nullptr;
    o.window = 1;
    o.sinks = 0x7fffffff;  // every key
    o.evict_first = L.own.row_groups == 1 ? 1 : 0;
    o.kv_scales = a->kv_scales;
    o.fp8_rope_off = a->kv_scales ? kDv : kFp8RopeOffset;
    e = L.own.mode == 7 ? launch_decode_rows(tm_q, a->q, o, true, s)
                        : launch_decode(tm_own_q, tm_own_kv, o, L.own.rpc, L.own.mode, s);
    if (e != cudaSuccess) return cuda_fail(e, "decode kernel launch");
  }
  MergeParams m;
  memset(&m, 0, sizeof m);
  m.total_rows = static_cast<int>(qrows);
  if (a->is_fp8) {
    m.prefix = MergeSide{p.spans, p.o_accum, p.lse_accum, 2 * L.pre.num_parts};
    m.own = MergeSide{reinterpret_cast<int32_t*>(ws + L.own_spans), reinterpret_cast<float*>(ws + L.own_o),
                      reinterpret_cast<float*>(ws + L.own_lse), 2 * L.own.num_parts};
    m.has_prefix = 1;
    m.rows = L.own.rows;
    m.problems = a->batch;
  } else {
    m.own = MergeSide{p.spans, p.o_accum, p.lse_accum, -1};
    m.rows = 128;
    m.problems = L.pre.num_problems;
  }
  m.out = a->out;
  m.lse = a->lse;
  e = launch_merge(m, s);
  if (e != cudaSuccess) return cuda_fail(e, "merge kernel launch");
  return ok();
}

mla_status mla_index_topk_workspace_size(int num_tokens, int block_table_stride, size_t* bytes) {
  if (!bytes) return fail(MLA_ERR_INVALID_ARG, "bytes is NULL");
  if (num_tokens < 0) return fail(MLA_ERR_INVALID_ARG, "num_tokens must be >= 0 (got %d)", num_tokens);
  if (block_table_stride < 1)
    return fail(MLA_ERR_INVALID_ARG, "block_table_stride must be >= 1 (got %d)", block_table_stride);
  *bytes = align256(static_cast<size_t>(num_tokens) * block_table_stride * kPageSize * sizeof(float));
  return ok();
}

mla_status mla_index_topk(const mla_index_topk_args* a, mla_stream_t stream) {
  if (!a) return fail(MLA_ERR_INVALID_ARG, "args is NULL");
  if (a->batch < 1) return fail(MLA_ERR_INVALID_ARG, "batch must be >= 1 (got %d)", a->batch);
  if (a->num_tokens < 0) return fail(MLA_ERR_INVALID_ARG, "num_tokens must be >= 0 (got %d)", a->num_tokens);
  if (a->h_idx < 8 || a->h_idx % 8 != 0 || a->h_idx > 256)
    return fail(MLA_ERR_UNSUPPORTED, "h_idx must be a multiple of 8 in [8, 256] (got %d)", a->h_idx);
  if (a->max_new_tokens < 1) return fail(MLA_ERR_INVALID_ARG, "max_new_tokens must be >= 1 (got %d)", a->max_new_tokens);
  if (static_cast<long long>(a->max_new_tokens) * a->h_idx > 256)
    return fail(MLA_ERR_UNSUPPORTED, "max_new_tokens * h_idx = %lld exceeds 256 rows per element",
                static_cast<long long>(a->max_new_tokens) * a->h_idx);
  if (a->topk < 1 || a->topk > 16384) return fail(MLA_ERR_UNSUPPORTED, "topk must be in [1, 16384] (got %d)", a->topk);
  if (a->page_size != kPageSize) return fail(MLA_ERR_UNSUPPORTED, "page_size must be 64 (got %d)", a->page_size);
  if (a->num_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages must be >= 1 (got %d)", a->num_pages);
  if (a->block_table_stride < 1)
    return fail(MLA_ERR_INVALID_ARG, "block_table_stride must be >= 1 (got %d)", a->block_table_stride);
  if (static_cast<long long>(a->block_table_stride) * kPageSize > (1ll << 31) - 1)
    return fail(MLA_ERR_UNSUPPORTED, "block_table_stride = %d exceeds 2^31 keys", a->block_table_stride);
  if (!a->q_codes) return fail(MLA_ERR_INVALID_ARG, "q_codes is NULL");
  if (!a->q_scales) return fail(MLA_ERR_INVALID_ARG, "q_scales is NULL");
  if (!a->weights) return fail(MLA_ERR_INVALID_ARG, "weights is NULL");
  if (!a->row_offsets) return fail(MLA_ERR_INVALID_ARG, "row_offsets is NULL");
  if (!a->k_codes) return fail(MLA_ERR_INVALID_ARG, "k_codes is NULL");
  if (!a->k_scales) return fail(MLA_ERR_INVALID_ARG, "k_scales is NULL");
  if (!a->block_table) return fail(MLA_ERR_INVALID_ARG, "block_table is NULL");
  if (!a->cache_seqlens) return fail(MLA_ERR_INVALID_ARG, "cache_seqlens is NULL");
  if (!a->indices) return fail(MLA_ERR_INVALID_ARG, "indices is NULL");
  if (!aligned(a->q_codes, 16)) return fail(MLA_ERR_INVALID_ARG, "q_codes is not 16-byte aligned");
  if (!aligned(a->k_codes, 16)) return fail(MLA_ERR_INVALID_ARG, "k_codes is not 16-byte aligned");
  size_t need = 0;
  mla_status st = mla_index_topk_workspace_size(a->num_tokens, a->block_table_stride, &need);
  if (st != MLA_OK) return st;
  if (a->num_tokens == 0) return ok();
  if (!a->workspace) return fail(MLA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
  if (a->workspace_bytes < need) return fail(MLA_ERR_WORKSPACE, "workspace_bytes = %zu < %zu needed", a->workspace_bytes, need);
  if (!aligned(a->workspace, 16)) return fail(MLA_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  uint32_t* status = nullptr;
  st = device_info(&status, nullptr);
  if (st != MLA_OK) return st;

  IndexParams p;
  memset(&p, 0, sizeof p);
  const int rows = a->max_new_tokens * a->h_idx;
  p.n_box = (rows + 15) & ~15;
  uint32_t cols = 32;
  while (cols < static_cast<uint32_t>(p.n_box)) cols <<= 1;
  p.tmem_cols = 2 * cols;
  CUtensorMap tm_q, tm_k;
  st = encode_e4m3_rows_map(&tm_q, a->q_codes, static_cast<long long>(a->num_tokens) * a->h_idx, p.n_box, "q_codes");
  if (st != MLA_OK) return st;
  st = encode_e4m3_rows_map(&tm_k, a->k_codes, static_cast<long long>(a->num_pages) * kPageSize, kPageSize, "k_codes");
  if (st != MLA_OK) return st;
  p.q_scales = a->q_scales;
  p.weights = a->weights;
  p.row_offsets = a->row_offsets;
  p.k_scales = a->k_scales;
  p.block_table = a->block_table;
  p.cache_seqlens = a->cache_seqlens;
  p.scores = static_cast<float*>(a->workspace);
  p.status = status;
  p.timeout_ns = watchdog_ns();
  p.width = static_cast<int64_t>(a->block_table_stride) * kPageSize;
  p.batch = a->batch;
  p.num_tokens = a->num_tokens;
  p.h_idx = a->h_idx;
  p.max_new = a->max_new_tokens;
  p.num_pages = a->num_pages;
  p.block_table_stride = a->block_table_stride;
  p.relu = a->relu ? 1 : 0;
  // key tiles per CTA: the run length that minimises the modelled time when
  // every element has the longest possible length -- whole waves of two CTAs
  // per SM, each costing its tiles plus about three tiles of set-up and
  // pipeline fill (a last, partly filled wave costs as much as a full one)
  {
    int sms = 0;
    st = device_info(nullptr, &sms);
    if (st != MLA_OK) return st;
    const long long max_tiles = (p.width + 127) / 128;
    const long long slots = 2ll * (sms > 0 ? sms : 1);
    long long best_cost = -1, best_tpc = 64;
    for (long long tpc = 4; tpc <= 64; ++tpc) {
      const long long ctas = static_cast<long long>(a->batch) * ((max_tiles + tpc - 1) / tpc);
      const long long waves = (ctas + slots - 1) / slots;
      const long long cost = waves * (tpc + 3);
      if (best_cost < 0 || cost < best_cost) {
        best_cost = cost;
        best_tpc = tpc;
      }
    }
    p.tiles_per_cta = static_cast<int>(best_tpc);
  }
  cudaError_t e = launch_index(tm_q, tm_k, p, a->topk, a->indices, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "indexer kernel launch");
  return ok();
}

mla_status mla_get_device_status(mla_stream_t stream, uint32_t* flags) {
  if (!flags) return fail(MLA_ERR_INVALID_ARG, "flags is NULL");
  uint32_t* status = nullptr;
  mla_status st = device_info(&status, nullptr);
  if (st != MLA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  uint32_t v = 0;
  e = cudaMemcpyAsync(&v, status, sizeof v, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(status, 0, sizeof v, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "reading the device status word");
  *flags = v;
  if (v & MLA_DEVICE_TIMEOUT) return fail(MLA_ERR_DEVICE_TIMEOUT, "a kernel wait exceeded its limit (status 0x%x)", v);
  if (v & MLA_DEVICE_BAD_PAGE)
    return fail(MLA_ERR_DEVICE_BOUNDS, "a block-table entry was outside [0, num_pages) (status 0x%x)", v);
  if (v & MLA_DEVICE_BAD_SCHEDULE)
    return fail(MLA_ERR_INVALID_ARG, "the schedule did not match the decode arguments (status 0x%x)", v);
  if (v & MLA_DEVICE_NO_ROOM)
    return fail(MLA_ERR_DEVICE_BOUNDS, "new tokens did not get their pages or slots (status 0x%x)", v);
  return ok();
}

}  // extern "C"
