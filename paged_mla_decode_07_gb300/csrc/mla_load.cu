// K11 — cached tokens of a batch as packed bf16 rows: what a chunked prefill
// reads before it projects the latents up.
//
// Row t belongs to request b, the last one with row_offsets[b] <= t, and is the
// token at position starts[b] + t - row_offsets[b] of it, looked up through the
// block table.  Its 576 values are what the row stands for: bf16 rows as they
// are, FP8 code * scale rounded to bf16 (the format's definition), FP4 code *
// scale, which is a bf16 number.
//
// Memory-bound: a row of 400 to 1152 bytes read and 1152 bytes written per
// token, behind four reads that depend on each other (the offsets, by a search 32
// requests wide, the start, the page, the row): a warp has one token, or two of
// long calls, in a grid that fills the chip several times over, so that the reads
// of many tokens overlap.  Lane k of a warp finds the row of its token k; then lane
// l holds dims 16 l .. 16 l + 15 and, up to lane 7, eight RoPE values.  110304
// tokens of FP8 rows take 40.0 us (5.0 TB/s; a copy of as many bytes 40.1), 30001
// of FP4 rows 17.5 (a launch alone 7.3); with four tokens a warp in a grid of eight
// blocks an SM 41.1 and 21.7, one token there 42.0 and 21.6.
#include "mla_device.cuh"
#include "mla_fp4.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kLoadWarps = 8;

template <int FMT>
struct Row {
  static constexpr int kBytes = FMT == MLA_CACHE_BF16        ? 2 * kDqk
                                : FMT == MLA_CACHE_FP8       ? kFp8RowBytes
                                : FMT == MLA_CACHE_FP8_TOKEN ? 640
                                                             : kFp4RowBytes;
  static constexpr int kRope = kBytes - 2 * (kDqk - kDv);
};

// The request of row t: the last b with row_offsets[b] <= t (the offsets of
// requests without tokens repeat).  All lanes.
__device__ __forceinline__ int request_of(const int32_t* __restrict__ offsets, int batch, int t, int lane) {
  int lo = 0, n = batch;  // in [lo, lo + n); offsets[lo] <= t
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool below = lane * step < n && __ldg(offsets + at) <= t;
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, below || lane == 0));
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

template <int FMT, int T>
__global__ void __launch_bounds__(kLoadWarps * 32) cache_load_kernel(const CacheLoadParams p) {
  const int lane = threadIdx.x & 31;
  const int total = min(__ldg(p.row_offsets + p.batch), p.num_tokens);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kLoadWarps * T;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kLoadWarps + (threadIdx.x >> 5)) * T; t0 < total; t0 += step) {
    // lane k finds the row of token k: its request, its page
    int b = request_of(p.row_offsets, p.batch, static_cast<int>(t0), lane);
    int64_t mine = -1;
    const int64_t t = t0 + lane;
    if (lane < T && t < total) {
      int first = __ldg(p.row_offsets + b), next = __ldg(p.row_offsets + b + 1);
      while (t >= next && b + 1 < p.batch) {
        ++b;
        first = next;
        next = __ldg(p.row_offsets + b + 1);
      }
      const int64_t pos = (p.starts ? __ldg(p.starts + b) : 0) + (t - first), page_at = pos / kPageSize;
      int page = -1;
      if (pos >= 0 && page_at < p.block_table_stride)
        page = __ldg(p.block_table + static_cast<int64_t>(b) * p.block_table_stride + page_at);
      if (page >= 0 && page < p.num_pages)
        mine = static_cast<int64_t>(page) * kPageSize + pos % kPageSize;
      else
        atomicOr(p.status, MLA_DEVICE_BAD_PAGE);
    }
    int64_t row[T];
#pragma unroll
    for (int k = 0; k < T; ++k) row[k] = __shfl_sync(0xffffffffu, mine, k);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 a[T], c[T], rope[T];
    float scale[T];
#pragma unroll
    for (int k = 0; k < T; ++k) {
      a[k] = c[k] = rope[k] = zero;
      scale[k] = 0.f;
      if (row[k] < 0) continue;
      const uint8_t* src = p.kvcache + row[k] * Row<FMT>::kBytes;
      if (FMT == MLA_CACHE_BF16) {
        a[k] = ld_global_nc_v4(src + 32 * lane);
        c[k] = ld_global_nc_v4(src + 32 * lane + 16);
      } else if (FMT == MLA_CACHE_FP4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(src) + lane);
        a[k].x = w.x;
        a[k].y = w.y;
        const uint32_t i = fp4_scale_index(__ldg(src + kFp4ScaleOffset + (lane >> 1)));
        scale[k] = __uint_as_float((i + kFp4ScaleMin) << 23);
      } else {
        a[k] = ld_global_nc_v4(src + 16 * lane);
        scale[k] = FMT == MLA_CACHE_FP8_TOKEN ? __ldg(p.kv_scales + row[k])
                                              : __ldg(reinterpret_cast<const float*>(src + kFp8ScaleOffset) + (lane >> 3));
      }
      if (lane < 8) rope[k] = ld_global_nc_v4(src + Row<FMT>::kRope + 16 * lane);
    }
#pragma unroll
    for (int k = 0; k < T; ++k) {
      if (t0 + k >= total) continue;
      uint4* dst = reinterpret_cast<uint4*>(p.out + (t0 + k) * (2 * kDqk));
      uint4 lo = a[k], hi = c[k];
      if (FMT == MLA_CACHE_FP4) {
        float v[8];
        fp4_floats(a[k].x, scale[k], v);
        lo = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        fp4_floats(a[k].y, scale[k], v);
        hi = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      } else if (FMT != MLA_CACHE_BF16) {
        auto pair = [&](uint32_t w, int half) { return e4m3x2_scaled_bf16x2((w >> (16 * half)) & 0xffffu, scale[k]); };
        lo = make_uint4(pair(a[k].x, 0), pair(a[k].x, 1), pair(a[k].y, 0), pair(a[k].y, 1));
        hi = make_uint4(pair(a[k].z, 0), pair(a[k].z, 1), pair(a[k].w, 0), pair(a[k].w, 1));
      }
      dst[2 * lane] = lo;
      dst[2 * lane + 1] = hi;
      if (lane < 8) dst[64 + lane] = rope[k];
    }
  }
}

template <int FMT>
cudaError_t launch(const CacheLoadParams& p, int sm_count, cudaStream_t stream) {
  // one token per warp until every warp of the grid has one
  const int64_t most = 64ll * sm_count;
  const bool two = p.num_tokens > most * kLoadWarps;
  const int64_t per = kLoadWarps * (two ? 2 : 1), need = (p.num_tokens + per - 1) / per;
  const unsigned grid = static_cast<unsigned>(need < most ? need : most);
  if (two)
    cache_load_kernel<FMT, 2><<<grid, kLoadWarps * 32, 0, stream>>>(p);
  else
    cache_load_kernel<FMT, 1><<<grid, kLoadWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_load(const CacheLoadParams& p, int sm_count, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  switch (p.format) {
    case MLA_CACHE_BF16: return launch<MLA_CACHE_BF16>(p, sm_count, stream);
    case MLA_CACHE_FP8: return launch<MLA_CACHE_FP8>(p, sm_count, stream);
    case MLA_CACHE_FP8_TOKEN: return launch<MLA_CACHE_FP8_TOKEN>(p, sm_count, stream);
    default: return launch<MLA_CACHE_FP4>(p, sm_count, stream);
  }
}

}  // namespace mla
