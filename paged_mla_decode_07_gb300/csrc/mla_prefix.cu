// K8 — the shared prefix of an FP8 cache as bf16 rows.
//
// A shared prefix is read under every block of 128 query rows, so its FP8 rows
// are turned into the values they stand for, bf16_rn(fp32(e4m3) * scale), once
// per call and not once per block: rows of 576 bf16 values in page order, the
// operand layout of the bf16 kernels.  One warp per token: lane l converts
// codes [16 l, 16 l + 16).  Memory-bound: 656 (640 + 4) bytes read and 1152
// written per token.
#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kRowWarps = 8;

__global__ void __launch_bounds__(kRowWarps * 32)
    prefix_rows_kernel(const uint8_t* __restrict__ kvcache, const float* __restrict__ kv_scales,
                       const int32_t* __restrict__ prefix_table, const int32_t* __restrict__ prefix_len,
                       int prefix_pages, int num_pages, uint8_t* __restrict__ rows, int32_t* __restrict__ table,
                       uint32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kRowWarps;
  const int64_t cap = static_cast<int64_t>(prefix_pages) * kPageSize;
  const int len = prefix_len[0];
  const int64_t n = len < cap ? len : cap;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5); t < n; t += warps) {
    const int lp = static_cast<int>(t / kPageSize);
    const int pg = __ldg(prefix_table + lp);
    const bool ok = pg >= 0 && pg < num_pages;
    if (t % kPageSize == 0 && lane == 0) {
      table[lp] = ok ? lp : -1;
      if (!ok) atomicOr(status, MLA_DEVICE_BAD_PAGE);
    }
    if (!ok) continue;
    const int64_t row = static_cast<int64_t>(pg) * kPageSize + t % kPageSize;
    const uint8_t* src = kvcache + row * (kv_scales ? 640 : kFp8RowBytes);
    const uint4 c = ld_global_nc_v4(src + 16 * lane);
    const float scale = kv_scales ? __ldg(kv_scales + row)
                                  : __ldg(reinterpret_cast<const float*>(src + kFp8ScaleOffset) + (lane >> 3));
    uint4* dst = reinterpret_cast<uint4*>(rows + t * (2 * kDqk));
    if (lane < 8) dst[64 + lane] = ld_global_nc_v4(src + (kv_scales ? kDv : kFp8RopeOffset) + 16 * lane);
    dst[2 * lane] = make_uint4(e4m3x2_scaled_bf16x2(c.x & 0xffffu, scale), e4m3x2_scaled_bf16x2(c.x >> 16, scale),
                               e4m3x2_scaled_bf16x2(c.y & 0xffffu, scale), e4m3x2_scaled_bf16x2(c.y >> 16, scale));
    dst[2 * lane + 1] = make_uint4(e4m3x2_scaled_bf16x2(c.z & 0xffffu, scale), e4m3x2_scaled_bf16x2(c.z >> 16, scale),
                                   e4m3x2_scaled_bf16x2(c.w & 0xffffu, scale), e4m3x2_scaled_bf16x2(c.w >> 16, scale));
  }
}

}  // namespace

cudaError_t launch_prefix_rows(const uint8_t* kvcache, const float* kv_scales, const int32_t* prefix_table,
                               const int32_t* prefix_len, int prefix_pages, int num_pages, void* rows, int32_t* table,
                               uint32_t* status, int sm_count, cudaStream_t stream) {
  const int64_t need = static_cast<int64_t>(prefix_pages) * kPageSize / kRowWarps;
  const int64_t most = 8ll * sm_count;
  prefix_rows_kernel<<<static_cast<unsigned>(need < most ? need : most), kRowWarps * 32, 0, stream>>>(
      kvcache, kv_scales, prefix_table, prefix_len, prefix_pages, num_pages, static_cast<uint8_t*>(rows), table, status);
  return cudaGetLastError();
}

}  // namespace mla
