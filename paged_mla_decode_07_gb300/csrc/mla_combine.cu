// K2 — merge split-KV partial results by their log-sum-exps.
//
// A problem whose keys were split over several parts has, per query row, one
// fp32 partial output o_i (already normalised by its own row sum) and its
// base-2 log-sum-exp lse_i.  The merged row is
//     L = log2 sum_i 2^{lse_i},   out = sum_i 2^{lse_i - L} o_i,   lse = L,
// the same rescaling that online softmax applies across tiles (Modular
// design-doc overview, section 6 "Matmul to Flash Attention"; the FlashMLA
// article, Design 5, pairs split-KV decode with a combine kernel launched
// with programmatic dependent launch).  Partials with lse = -inf contribute
// nothing; a problem with no keys at all gets out = 0, lse = -inf.
//
// One warp per output row; lane l owns dims [16l, 16l + 16).
#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kRowsPerBlock = 4;
constexpr int kFastSplits = 4;  // pieces merged with all loads in flight at once

__global__ void __launch_bounds__(kRowsPerBlock * 32) combine_kernel(const CombineParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t grow = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 5);
  if (grow >= static_cast<int64_t>(p.num_problems) * p.rows) return;
  const int prob = static_cast<int>(grow / p.rows);
  const int r = static_cast<int>(grow % p.rows);
  const int base = p.num_splits[prob];
  const int n = p.num_splits[prob + 1] - base;
  if (n == 0) {
    // a single piece wrote the output directly; a problem without any tile
    // (no keys) was touched by no part: its output is 0, its lse -inf
    if (problem_tiles(p.cache_seqlens, prob, p.s_q, p.topk) > 0) return;
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + grow * kDv + lane * 16;
    const uint4 z = make_uint4(0, 0, 0, 0);
    reinterpret_cast<uint4*>(out)[0] = z;
    reinterpret_cast<uint4*>(out)[1] = z;
    if (lane == 0) p.lse[grow] = -__int_as_float(0x7f800000);
    return;
  }
  if (base < 0 || n < 2 || base + n > p.max_slots) {
    if (lane == 0) atomicOr(p.status, MLA_DEVICE_BAD_SCHEDULE);
    return;
  }
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + grow * kDv + lane * 16;

  if (n <= kFastSplits) {
    // few pieces (the common case): every load is issued before any is used,
    // so the merge costs two memory round trips instead of one per piece
    float l[kFastSplits];
#pragma unroll
    for (int i = 0; i < kFastSplits; ++i)
      l[i] = i < n ? p.lse_accum[static_cast<int64_t>(base + i) * p.rows + r] : -__int_as_float(0x7f800000);
    float4 x[kFastSplits][4];
#pragma unroll
    for (int i = 0; i < kFastSplits; ++i) {
      if (i < n) {
        const float4* src = reinterpret_cast<const float4*>(p.o_accum + (static_cast<int64_t>(base + i) * p.rows + r) * kDv +
                                                            lane * 16);
#pragma unroll
        for (int v = 0; v < 4; ++v) x[i][v] = src[v];
      }
    }
    float mxf = l[0];
#pragma unroll
    for (int i = 1; i < kFastSplits; ++i) mxf = fmaxf(mxf, l[i]);
    float acc[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    float Lf = -__int_as_float(0x7f800000);
    if (mxf != -__int_as_float(0x7f800000)) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kFastSplits; ++i)
        if (i < n) sum += exp2f(l[i] - mxf);
      Lf = mxf + log2f(sum);
#pragma unroll
      for (int i = 0; i < kFastSplits; ++i) {
        if (i < n) {
          const float w = exp2f(l[i] - Lf);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            acc[4 * v + 0] += w * x[i][v].x;
            acc[4 * v + 1] += w * x[i][v].y;
            acc[4 * v + 2] += w * x[i][v].z;
            acc[4 * v + 3] += w * x[i][v].w;
          }
        }
      }
    }
    uint4 o0, o1;
    o0.x = pack_bf16x2(acc[0], acc[1]);
    o0.y = pack_bf16x2(acc[2], acc[3]);
    o0.z = pack_bf16x2(acc[4], acc[5]);
    o0.w = pack_bf16x2(acc[6], acc[7]);
    o1.x = pack_bf16x2(acc[8], acc[9]);
    o1.y = pack_bf16x2(acc[10], acc[11]);
    o1.z = pack_bf16x2(acc[12], acc[13]);
    o1.w = pack_bf16x2(acc[14], acc[15]);
    reinterpret_cast<uint4*>(out)[0] = o0;
    reinterpret_cast<uint4*>(out)[1] = o1;
    if (lane == 0) p.lse[grow] = Lf;
    return;
  }

  float mx = -__int_as_float(0x7f800000);
  for (int i = lane; i < n; i += 32) mx = fmaxf(mx, p.lse_accum[static_cast<int64_t>(base + i) * p.rows + r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (n <= 0 || mx == -__int_as_float(0x7f800000)) {
    const uint4 z = make_uint4(0, 0, 0, 0);
    reinterpret_cast<uint4*>(out)[0] = z;
    reinterpret_cast<uint4*>(out)[1] = z;
    if (lane == 0) p.lse[grow] = -__int_as_float(0x7f800000);
    return;
  }
  float s = 0.f;
  for (int i = lane; i < n; i += 32) s += exp2f(p.lse_accum[static_cast<int64_t>(base + i) * p.rows + r] - mx);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float L = mx + log2f(s);

  float acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  for (int i = 0; i < n; ++i) {
    const int64_t slot_row = static_cast<int64_t>(base + i) * p.rows + r;
    const float w = exp2f(p.lse_accum[slot_row] - L);
    const float4* src = reinterpret_cast<const float4*>(p.o_accum + slot_row * kDv + lane * 16);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float4 x = src[v];
      acc[4 * v + 0] += w * x.x;
      acc[4 * v + 1] += w * x.y;
      acc[4 * v + 2] += w * x.z;
      acc[4 * v + 3] += w * x.w;
    }
  }
  uint4 o0, o1;
  o0.x = pack_bf16x2(acc[0], acc[1]);
  o0.y = pack_bf16x2(acc[2], acc[3]);
  o0.z = pack_bf16x2(acc[4], acc[5]);
  o0.w = pack_bf16x2(acc[6], acc[7]);
  o1.x = pack_bf16x2(acc[8], acc[9]);
  o1.y = pack_bf16x2(acc[10], acc[11]);
  o1.z = pack_bf16x2(acc[12], acc[13]);
  o1.w = pack_bf16x2(acc[14], acc[15]);
  reinterpret_cast<uint4*>(out)[0] = o0;
  reinterpret_cast<uint4*>(out)[1] = o1;
  if (lane == 0) p.lse[grow] = L;
}

// ---------------------------------------------------------------------------
// Merges of windowed and shared-prefix decode
// ---------------------------------------------------------------------------
// A block merges one row with all its 128 threads, thread t owning dims
// [4 t, 4 t + 4) and eight pieces' 2 KB lines in flight, or four rows with a
// warp each.  The first suits few rows in many pieces (a small batch is cut
// over all SMs: 96 rows of 17 pieces take ~5 us less), the second many rows in
// few (12288 rows of two pieces take 5 us less).  Bound by latency (spans,
// log-sum-exps, values: three dependent reads), and by the partials' bytes
// where there are many rows.
constexpr int kMergeThreads = 128;
constexpr float kMergeNegInf = -__builtin_huge_valf();

// The pieces of problem `prob` of a side: n of them, the first in slot `slot`,
// the others in those of the parts behind it.  n = -1: a part held the problem
// whole and wrote its output.
struct Pieces {
  int n, slot;
  __device__ __forceinline__ int at(int i) const { return i == 0 ? slot : 2 * ((slot >> 1) + i); }
};
__device__ __forceinline__ Pieces find_pieces(const MergeSide& m, int prob) {
  const int2 s = reinterpret_cast<const int2*>(m.spans)[prob];
  const int n = s.y - (s.x >> 1) + 1;
  if (n == 1) return m.whole_base < 0 ? Pieces{-1, 0} : Pieces{1, m.whole_base + prob};
  return Pieces{n, s.x};
}

// Merges the pieces of one row with all threads of the block.
template <class At>
__device__ __forceinline__ void merge_row_block(int n, At at, __nv_bfloat16* out, float* lse) {
  const int lane = threadIdx.x & 31;
  auto lse_at = [&](int i) { return *at(i).second; };
  const float first = lane < n ? lse_at(lane) : kMergeNegInf;  // pieces 0..31, one per lane
  float mx = first;
  for (int i = lane + 32; i < n; i += 32) mx = max_nan(mx, lse_at(i));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float L = kMergeNegInf;
  if (mx != kMergeNegInf) {
    float sum = lane < n ? exp2f(first - mx) : 0.f;
    for (int i = lane + 32; i < n; i += 32) sum += exp2f(lse_at(i) - mx);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    L = mx + log2f(sum);
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int m = min(32, n - i0);
      // weight of piece i0 + lane (0 past the end and for pieces without keys)
      const float w = lane < m ? exp2f((i0 == 0 ? first : lse_at(i0 + lane)) - L) : 0.f;
#pragma unroll 1
      for (int k0 = 0; k0 < m; k0 += 8) {
        // (values of a piece without keys for this row are not there)
        float4 v[8];
        float wk[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          wk[k] = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
          if (k0 + k < m && wk[k] != 0.f) v[k] = at(i0 + k0 + k).first[threadIdx.x];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k0 + k < m && wk[k] != 0.f) {
            acc.x += wk[k] * v[k].x;
            acc.y += wk[k] * v[k].y;
            acc.z += wk[k] * v[k].z;
            acc.w += wk[k] * v[k].w;
          }
        }
      }
    }
  }
  reinterpret_cast<uint2*>(out)[threadIdx.x] = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
  if (threadIdx.x == 0) *lse = L;
}

// Merges the pieces of one row with one warp: lane l owns dims 128 v + 4 l .. + 3.
template <class At>
__device__ __forceinline__ void merge_row_warp(int n, At at, __nv_bfloat16* out, float* lse) {
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 31;
  float mx = kMergeNegInf;
  for (int i = lane; i < n; i += 32) mx = max_nan(mx, *at(i).second);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float4 acc[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  float L = kMergeNegInf;
  if (mx != kMergeNegInf) {
    float sum = 0.f;
    for (int i = lane; i < n; i += 32) sum += exp2f(*at(i).second - mx);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    L = mx + log2f(sum);
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kAhead) {
      float4 x[kAhead][4];
      float w[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        w[i] = kMergeNegInf;
        if (i0 + i < n) {
          const auto piece = at(i0 + i);
          w[i] = *piece.second;
#pragma unroll
          for (int v = 0; v < 4; ++v) x[i][v] = piece.first[32 * v + lane];
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (i0 + i >= n) break;
        const float wi = exp2f(w[i] - L);
        if (wi == 0.f) continue;  // (values of a piece without keys for this row are not there)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          acc[v].x += wi * x[i][v].x;
          acc[v].y += wi * x[i][v].y;
          acc[v].z += wi * x[i][v].z;
          acc[v].w += wi * x[i][v].w;
        }
      }
    }
  }
#pragma unroll
  for (int v = 0; v < 4; ++v)
    reinterpret_cast<uint2*>(out)[32 * v + lane] =
        make_uint2(pack_bf16x2(acc[v].x, acc[v].y), pack_bf16x2(acc[v].z, acc[v].w));
  if (lane == 0) *lse = L;
}

struct PiecePtr {
  const float4* first;   // the piece's 512 values
  const float* second;   // its log-sum-exp
};

// grid: (row blocks of a problem, problems); WARP_ROWS: four rows per block, a
// warp each (then an element's rows are a multiple of four where there is a
// prefix, so that the four lie in one block of its rows).
template <bool WARP_ROWS>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const MergeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int prob = blockIdx.y;
  const int r = blockIdx.x * (WARP_ROWS ? 4 : 1) + (WARP_ROWS ? threadIdx.x >> 5 : 0);
  const int64_t row = static_cast<int64_t>(prob) * p.rows + r;
  const Pieces own_pieces = find_pieces(p.own, prob);
  Pieces prefix_pieces{0, 0};
  if (r >= p.rows || row >= p.total_rows) return;
  if (p.has_prefix) prefix_pieces = find_pieces(p.prefix, static_cast<int>(row / 128));
  const int n0 = prefix_pieces.n, n1 = own_pieces.n;
  if (n1 < 0) return;  // one part held the problem and wrote its rows
  auto at = [&](int i) {
    const bool in_prefix = i < n0;
    const MergeSide& m = in_prefix ? p.prefix : p.own;
    const int slot = in_prefix ? prefix_pieces.at(i) : own_pieces.at(i - n0);
    const int64_t s = in_prefix ? static_cast<int64_t>(slot) * 128 + row % 128 : static_cast<int64_t>(slot) * p.rows + r;
    return PiecePtr{reinterpret_cast<const float4*>(m.o + s * kDv), m.lse + s};
  };
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + row * kDv;
  if (WARP_ROWS)
    merge_row_warp(n0 + n1, at, out, p.lse + row);
  else
    merge_row_block(n0 + n1, at, out, p.lse + row);
}

}  // namespace

cudaError_t launch_merge(const MergeParams& p, cudaStream_t stream) {
  // rows enough to fill the chip four to a block, in few pieces each
  const bool warp_rows = p.total_rows >= 2048 && (!p.has_prefix || p.rows % 4 == 0);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(warp_rows ? (p.rows + 3) / 4 : p.rows), static_cast<unsigned>(p.problems));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return warp_rows ? cudaLaunchKernelEx(&cfg, merge_kernel<true>, p) : cudaLaunchKernelEx(&cfg, merge_kernel<false>, p);
}

cudaError_t launch_combine(const CombineParams& p, cudaStream_t stream, bool pdl) {
  const int64_t rows = static_cast<int64_t>(p.num_problems) * p.rows;
  const unsigned grid = static_cast<unsigned>((rows + kRowsPerBlock - 1) / kRowsPerBlock);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kRowsPerBlock * 32);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, combine_kernel, p);
}

}  // namespace mla
