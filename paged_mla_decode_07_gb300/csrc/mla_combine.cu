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

// Merges of windowed and shared-prefix decode, where a few rows may have many
// pieces (a small batch is cut over all SMs): one block of 128 threads per
// row, thread t owning dims [4 t, 4 t + 4), so that a row's pieces are read in
// whole 2 KB lines with eight in flight per thread; the 32 log-sum-exps of a
// round are one load of every warp and their weights reach the threads by
// shuffles.  Bound by latency for small batches (slots, log-sum-exps, values:
// three dependent reads) and by the partials' bytes for large ones: 96 rows of
// 17 pieces take ~5 us less than with a warp per row that reads piece by piece.
constexpr int kMergeThreads = 128;
constexpr float kMergeNegInf = -__builtin_huge_valf();

// Merges n pieces of one row; lse_at(i) and values_at(i) name piece i.
template <class LseAt, class ValuesAt>
__device__ __forceinline__ void merge_row(int n, LseAt lse_at, ValuesAt values_at, __nv_bfloat16* out, float* lse) {
  const int lane = threadIdx.x & 31;
  const float first = lane < n ? lse_at(lane) : kMergeNegInf;  // pieces 0..31, one per lane
  float mx = first;
  for (int i = lane + 32; i < n; i += 32) mx = fmaxf(mx, lse_at(i));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
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
        float4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k0 + k < m) v[k] = values_at(i0 + k0 + k)[threadIdx.x];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
          if (k0 + k < m) {
            acc.x += wk * v[k].x;
            acc.y += wk * v[k].y;
            acc.z += wk * v[k].z;
            acc.w += wk * v[k].w;
          }
        }
      }
    }
  }
  reinterpret_cast<uint2*>(out)[threadIdx.x] = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
  if (threadIdx.x == 0) *lse = L;
}

// Windowed decode: a problem in one piece wrote its rows itself; one without
// keys has none.
__global__ void __launch_bounds__(kMergeThreads) window_combine_kernel(const CombineParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int prob = blockIdx.x / p.rows, r = blockIdx.x % p.rows;
  const int base = p.num_splits[prob], n = p.num_splits[prob + 1] - base;
  if (n == 0 && p.cache_seqlens[prob] > 0) return;
  if (base < 0 || n < 0 || n == 1 || base + n > p.max_slots) {
    if (threadIdx.x == 0) atomicOr(p.status, MLA_DEVICE_BAD_SCHEDULE);
    return;
  }
  const int64_t at = static_cast<int64_t>(base) * p.rows + r;
  merge_row(
      n, [&](int i) { return p.lse_accum[at + static_cast<int64_t>(i) * p.rows]; },
      [&](int i) { return reinterpret_cast<const float4*>(p.o_accum + (at + static_cast<int64_t>(i) * p.rows) * kDv); },
      reinterpret_cast<__nv_bfloat16*>(p.out) + static_cast<int64_t>(blockIdx.x) * kDv, p.lse + blockIdx.x);
}

// Shared-prefix decode: a row's pieces lie in two runs of slots, the prefix
// under its block of 128 rows and its element's own keys, merged as one list.
// An element without own keys has none of the second, an empty prefix none of
// the first.
__global__ void __launch_bounds__(kMergeThreads) prefix_combine_kernel(const PrefixCombineParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int row = blockIdx.x;
  const int elem = row / p.rows, r = row % p.rows;
  const int pp = row / 128;
  const int op = elem * p.blocks_per_elem + r / p.block_rows;
  const int base0 = p.prefix_splits[pp], n0 = p.prefix_splits[pp + 1] - base0;
  // (both kinds may come from one schedule: the own slots count from the first own problem's)
  const int base1 = p.own_splits[op] - p.own_splits[0], n1 = p.own_splits[op + 1] - p.own_splits[op];
  if (base0 < 0 || n0 < 0 || base0 + n0 > p.prefix_slots || base1 < 0 || n1 < 0 || base1 + n1 > p.own_slots) {
    if (threadIdx.x == 0) atomicOr(p.status, MLA_DEVICE_BAD_SCHEDULE);
    return;
  }
  const int64_t at0 = static_cast<int64_t>(base0) * 128 + row % 128;
  const int64_t at1 = static_cast<int64_t>(base1) * p.block_rows + r % p.block_rows;
  merge_row(
      n0 + n1,
      [&](int i) {
        return i < n0 ? p.prefix_lse[at0 + static_cast<int64_t>(i) * 128]
                      : p.own_lse[at1 + static_cast<int64_t>(i - n0) * p.block_rows];
      },
      [&](int i) {
        return reinterpret_cast<const float4*>(i < n0 ? p.prefix_o + (at0 + static_cast<int64_t>(i) * 128) * kDv
                                                      : p.own_o + (at1 + static_cast<int64_t>(i - n0) * p.block_rows) * kDv);
      },
      reinterpret_cast<__nv_bfloat16*>(p.out) + static_cast<int64_t>(row) * kDv, p.lse + row);
}

template <class Params>
cudaError_t launch_merge(void (*kernel)(const Params), const Params& p, int64_t rows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_prefix_combine(const PrefixCombineParams& p, cudaStream_t stream) {
  return launch_merge(prefix_combine_kernel, p, p.total_rows, stream);
}

cudaError_t launch_window_combine(const CombineParams& p, cudaStream_t stream) {
  return launch_merge(window_combine_kernel, p, static_cast<int64_t>(p.num_problems) * p.rows, stream);
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
