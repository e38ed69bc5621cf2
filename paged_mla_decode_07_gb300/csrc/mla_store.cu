// K3 — FP8 KV-cache write: new tokens (576 bf16 values each) quantised into
// the 656-byte cache row and written through the block table.
//
// The row format follows the FlashMLA article (Design 2): the 512 NoPE dims
// become float8_e4m3 codes in four 1 x 128 tiles, each with one float32
// scale = amax / 448 (1 for an all-zero tile), code = E4M3 of x / scale
// rounded to nearest even and saturated at 448; the 64 RoPE dims are copied
// as bf16.  Placement follows the MAX kernels summary (KV-cache store): the
// new tokens of batch element b, rows input_row_offsets[b] ..
// input_row_offsets[b+1]-1 of x, go to logical positions cache_lengths[b] +
// i, i.e. page block_table[b][pos / 64], slot pos % 64.
//
// One warp per token: lane l holds NoPE dims [16l, 16l+16) (a tile is eight
// lanes; its amax is a three-step shuffle), lanes 0..7 the RoPE dims.  Each
// lane reads 32 + 16 bytes and writes 16 + 16 bytes with 16-byte accesses.
// Memory-bound: 1152 bytes read and 656 written per token.
#include <cuda_bf16.h>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kStoreWarps = 8;  // warps per block

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two floats -> two E4M3 codes (round to nearest even, saturating), low byte = lo.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Quantise one token (this lane's 16 NoPE values a, c and, for lanes 0..7,
// 8 RoPE values rp) into the row at dst.
__device__ __forceinline__ void store_row(uint8_t* dst, const uint4 a, const uint4 c, const uint4 rp, int lane) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float scale = amax > 0.f ? __fdiv_rn(amax, 448.0f) : 1.0f;
  uint32_t code[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    code[i] = e4m3x2(__fdiv_rn(v[4 * i], scale), __fdiv_rn(v[4 * i + 1], scale)) |
              (e4m3x2(__fdiv_rn(v[4 * i + 2], scale), __fdiv_rn(v[4 * i + 3], scale)) << 16);
  *reinterpret_cast<uint4*>(dst + 16 * lane) = make_uint4(code[0], code[1], code[2], code[3]);
  // scales: tile t is held by lanes 8t .. 8t+7
  const float s0 = __shfl_sync(0xffffffffu, scale, 0), s1 = __shfl_sync(0xffffffffu, scale, 8);
  const float s2 = __shfl_sync(0xffffffffu, scale, 16), s3 = __shfl_sync(0xffffffffu, scale, 24);
  if (lane == 0)
    *reinterpret_cast<uint4*>(dst + kFp8ScaleOffset) =
        make_uint4(__float_as_uint(s0), __float_as_uint(s1), __float_as_uint(s2), __float_as_uint(s3));
  if (lane < 8) *reinterpret_cast<uint4*>(dst + kFp8RopeOffset + 16 * lane) = rp;
}

// Each warp takes a contiguous range of token rows (one search for its first
// batch element, then advanced as rows cross element boundaries) and handles
// two rows per step, loading both rows before resolving their pages so the
// loads overlap the block-table lookups.
__global__ void __launch_bounds__(kStoreWarps * 32)
    fp8_store_kernel(const uint16_t* __restrict__ x, int num_tokens, const int32_t* __restrict__ row_offsets,
                     const int32_t* __restrict__ cache_lengths, int batch, const int32_t* __restrict__ block_table,
                     int block_table_stride, uint8_t* __restrict__ kvcache, int num_pages, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kStoreWarps;
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * kStoreWarps + (threadIdx.x >> 5);
  const int64_t per = (num_tokens + warps - 1) / warps;
  const int r0 = static_cast<int>(wid * per);
  const int r1 = static_cast<int>(((static_cast<int64_t>(r0) + per < num_tokens) ? static_cast<int64_t>(r0) + per : static_cast<int64_t>(num_tokens)));
  if (r0 >= r1) return;
  // batch element of row r0: the last b with row_offsets[b] <= r0
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(row_offsets + mid) <= r0)
      lo = mid;
    else
      hi = mid - 1;
  }
  int b = lo;
  int off_b = __ldg(row_offsets + b), off_n = __ldg(row_offsets + b + 1), len_b = __ldg(cache_lengths + b);
  // destination of row r (advances b while r is past the element's rows)
  auto dest = [&](int r) -> uint8_t* {
    while (r >= off_n && b + 1 < batch) {
      ++b;
      off_b = off_n;
      off_n = __ldg(row_offsets + b + 1);
      len_b = __ldg(cache_lengths + b);
    }
    const int64_t pos = static_cast<int64_t>(len_b) + (r - off_b);
    const int64_t blk = pos / kPageSize;
    const int page = (pos >= 0 && blk < block_table_stride)
                         ? __ldg(block_table + static_cast<int64_t>(b) * block_table_stride + blk)
                         : -1;
    if (page < 0 || page >= num_pages) {
      if (lane == 0) atomicOr(status, MLA_DEVICE_BAD_PAGE);
      return nullptr;
    }
    return kvcache + (static_cast<int64_t>(page) * kPageSize + pos % kPageSize) * kFp8RowBytes;
  };
  for (int r = r0; r < r1; r += 2) {
    const bool two = r + 1 < r1;
    const uint16_t* s0 = x + static_cast<int64_t>(r) * kDqk;
    const uint16_t* s1 = s0 + kDqk;
    const uint4 a0 = ld_global_nc_v4(s0 + 16 * lane), c0 = ld_global_nc_v4(s0 + 16 * lane + 8);
    const uint4 p0 = lane < 8 ? ld_global_nc_v4(s0 + kDv + 8 * lane) : make_uint4(0, 0, 0, 0);
    uint4 a1 = make_uint4(0, 0, 0, 0), c1 = a1, p1 = a1;
    if (two) {
      a1 = ld_global_nc_v4(s1 + 16 * lane);
      c1 = ld_global_nc_v4(s1 + 16 * lane + 8);
      if (lane < 8) p1 = ld_global_nc_v4(s1 + kDv + 8 * lane);
    }
    uint8_t* d0 = dest(r);
    uint8_t* d1 = two ? dest(r + 1) : nullptr;
    if (d0) store_row(d0, a0, c0, p0, lane);
    if (d1) store_row(d1, a1, c1, p1, lane);
  }
}

// ---------------------------------------------------------------------------
// K7 — store through a slot map: token i (512 latent and 64 RoPE values from
// two row-strided tensors) into cache row slots[i], in any row format.  The
// token's place is one read instead of the search and table lookup above.
// Memory-bound: 1152 bytes read and 1152, 656 or 644 written per token.
// ---------------------------------------------------------------------------
// Slot of token r, or -1 (padding, or a slot outside the cache, which is flagged).
__device__ __forceinline__ int slot_of(const SlotStoreParams& p, int r, bool flag) {
  const int s = __ldg(p.slots + r);
  if (s >= p.num_slots) {
    if (flag) atomicOr(p.status, MLA_DEVICE_BAD_PAGE);
    return -1;
  }
  return s < 0 ? -1 : s;
}

// Codes of 16 values at one scale, E4M3 of the correctly rounded x / scale.
// With r = RN(1 / scale), q0 = RN(x r) is within two units of the last place,
// one step q + r (x - q scale) brings it within one and a second one gives the
// correctly rounded quotient (Markstein 1990, theorem on division with a
// correctly rounded reciprocal): five instructions per value where the divide
// takes about ten, which bounds this kernel.  Remainders are exact while
// x 2^-48 is above the subnormals, for every x whose code is not 0 while
// scale >= 2^-90; scales outside [2^-90, 2^120] (infinities and NaN among
// them) divide.  The remainder is taken as q scale - x: it is +0 for x = -0 and
// for x = +0, so q - r (+0) has the sign of q, as the quotient does (with
// x - q scale, q + r (+0) would turn -0 into +0, and the code's sign with it).
__device__ __forceinline__ uint4 quantise16(const float (&v)[16], float scale) {
  float y[16];
  if (scale >= 8.077935669463161e-28f && scale <= 1.329227995784916e36f) {
    const float r = __frcp_rn(scale);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float q = v[i] * r;
      q = fmaf(-r, fmaf(q, scale, -v[i]), q);
      y[i] = fmaf(-r, fmaf(q, scale, -v[i]), q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = __fdiv_rn(v[i], scale);
  }
  uint32_t code[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) code[i] = e4m3x2(y[4 * i], y[4 * i + 1]) | (e4m3x2(y[4 * i + 2], y[4 * i + 3]) << 16);
  return make_uint4(code[0], code[1], code[2], code[3]);
}

// One token into its row: codes, RoPE values, and the scale of each 128
// values in the row or of all 512 at *scale_out.
template <bool TOKEN_SCALE>
__device__ __forceinline__ void store_slot_row(uint8_t* dst, float* scale_out, const uint4 a, const uint4 c,
                                               const uint4 rp, int lane) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
  for (int o = TOKEN_SCALE ? 16 : 4; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float scale = amax > 0.f ? __fdiv_rn(amax, 448.0f) : 1.0f;
  *reinterpret_cast<uint4*>(dst + 16 * lane) = quantise16(v, scale);
  if (TOKEN_SCALE) {
    if (lane == 0) *scale_out = scale;
  } else if ((lane & 7) == 0) {
    *reinterpret_cast<float*>(dst + kFp8ScaleOffset + (lane >> 1)) = scale;
  }
  if (lane < 8) *reinterpret_cast<uint4*>(dst + (TOKEN_SCALE ? kDv : kFp8RopeOffset) + 16 * lane) = rp;
}

// FP8 rows, one warp per token at a time, the next token's values loaded
// while this one is quantised.
template <bool TOKEN_SCALE>
__global__ void __launch_bounds__(kStoreWarps * 32) slot_store_fp8_kernel(const SlotStoreParams p) {
  constexpr int kRow = TOKEN_SCALE ? 640 : kFp8RowBytes;
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * kStoreWarps;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 a = zero, c = zero, rp = zero;
  int slot = -1;
  auto load = [&](int64_t r) {
    slot = slot_of(p, static_cast<int>(r), lane == 0);
    const uint16_t* s = p.latent + r * p.latent_stride + 16 * lane;
    a = ld_global_nc_v4(s);
    c = ld_global_nc_v4(s + 8);
    if (lane < 8) rp = ld_global_nc_v4(p.rope + r * p.rope_stride + 8 * lane);
  };
  int64_t r = static_cast<int64_t>(blockIdx.x) * kStoreWarps + (threadIdx.x >> 5);
  if (r < p.num_tokens) load(r);
#pragma unroll 1
  while (r < p.num_tokens) {
    const uint4 a0 = a, c0 = c, rp0 = rp;
    const int slot0 = slot;
    r += warps;
    if (r < p.num_tokens) load(r);
    if (slot0 >= 0)
      store_slot_row<TOKEN_SCALE>(p.kvcache + static_cast<int64_t>(slot0) * kRow,
                                  TOKEN_SCALE ? p.kv_scales + slot0 : nullptr, a0, c0, rp0, lane);
  }
}

// bf16 rows, copied as they are: a warp takes T consecutive tokens at a time,
// all loads issued before the first store.  Long stores run at the copy's pace
// only if neighbouring rows are in flight together (65535 tokens alone, the
// 151 MB take 26.5 us at T = 4, 28.7 at T = 1 and 39 with the 16-byte units of
// all rows dealt out grid-wide; a plain copy of as many bytes takes 24.7).
template <int T>
__global__ void __launch_bounds__(kStoreWarps * 32) slot_store_bf16_kernel(const SlotStoreParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kStoreWarps * T;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kStoreWarps + (threadIdx.x >> 5)) * T; t0 < p.num_tokens;
       t0 += step) {
    uint4 a[T], c[T], rp[T];
    int slot[T];
#pragma unroll
    for (int k = 0; k < T; ++k) {
      slot[k] = -1;
      if (t0 + k >= p.num_tokens) continue;
      slot[k] = slot_of(p, static_cast<int>(t0) + k, lane == 0);
      const uint16_t* s = p.latent + (t0 + k) * p.latent_stride + 8 * lane;
      a[k] = ld_global_nc_v4(s);
      c[k] = ld_global_nc_v4(s + 256);
      if (lane < 8) rp[k] = ld_global_nc_v4(p.rope + (t0 + k) * p.rope_stride + 8 * lane);
    }
#pragma unroll
    for (int k = 0; k < T; ++k) {
      if (slot[k] < 0) continue;
      uint4* dst = reinterpret_cast<uint4*>(p.kvcache + static_cast<int64_t>(slot[k]) * (2 * kDqk));
      dst[lane] = a[k];
      dst[32 + lane] = c[k];
      if (lane < 8) dst[64 + lane] = rp[k];
    }
  }
}

}  // namespace

cudaError_t launch_slot_store(const SlotStoreParams& p, int sm_count, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  const int64_t max_grid = sm_count * 8;
  const int threads = kStoreWarps * 32;
  // one token per warp until every warp of a full grid has one
  const bool four = !p.is_fp8 && p.num_tokens > max_grid * kStoreWarps;
  const int per_block = kStoreWarps * (four ? 4 : 1);
  const int64_t need = (static_cast<int64_t>(p.num_tokens) + per_block - 1) / per_block;
  const unsigned grid = static_cast<unsigned>(need < max_grid ? need : max_grid);
  if (p.is_fp8 && p.kv_scales) {
    slot_store_fp8_kernel<true><<<grid, threads, 0, stream>>>(p);
  } else if (p.is_fp8) {
    slot_store_fp8_kernel<false><<<grid, threads, 0, stream>>>(p);
  } else if (four) {
    slot_store_bf16_kernel<4><<<grid, threads, 0, stream>>>(p);
  } else {
    slot_store_bf16_kernel<1><<<grid, threads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_fp8_cache_store(const uint16_t* x, int num_tokens, const int32_t* row_offsets,
                                   const int32_t* cache_lengths, int batch, const int32_t* block_table,
                                   int block_table_stride, uint8_t* kvcache, int num_pages, uint32_t* status,
                                   int sm_count, cudaStream_t stream) {
  if (num_tokens == 0) return cudaSuccess;
  const int blocks_needed = (num_tokens + kStoreWarps - 1) / kStoreWarps;
  const int grid = blocks_needed < sm_count * 8 ? blocks_needed : sm_count * 8;
  fp8_store_kernel<<<grid, kStoreWarps * 32, 0, stream>>>(x, num_tokens, row_offsets, cache_lengths, batch,
                                                           block_table, block_table_stride, kvcache, num_pages,
                                                           status);
  return cudaGetLastError();
}

}  // namespace mla
