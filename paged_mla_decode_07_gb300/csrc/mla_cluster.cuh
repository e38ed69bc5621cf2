// Small windowed calls: a problem's pages are shared out over the CTAs of one
// thread-block cluster, and their results are merged through distributed shared
// memory, without a schedule, partial results in global memory or a second
// kernel (4 elements of 10 pages, 16 rows: bf16 11.9 us for 13.8, FP8 13.1 for
// 14.4).
#pragma once

#include "mla_device.cuh"
#include "mla_internal.h"
#include "mla_schedule.cuh"

namespace mla {

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// This CTA's share of the pages of problem `prob`.
__device__ __forceinline__ PartRecord cluster_share(const DecodeParams& p, int prob) {
  const int64_t n = key_walk(p.cache_seqlens[prob], p.s_q, p.window, p.sinks, p.block_table_stride).pages +
                    (p.prefix_len ? pages_of(p.prefix_len[0], p.prefix_pages) : 0);
  const int k = static_cast<int>(cluster_ctarank());
  return PartRecord{prob, static_cast<int>(n * k / p.cluster), prob, static_cast<int>(n * (k + 1) / p.cluster)};
}

// What a kernel keeps in shared memory for the merge, at the same place in
// every CTA: the byte offset of its rows from `base`, and their lse.
struct ClusterSide {
  const unsigned char* base;
  const int* o_at;   // normalised rows o [rows][512] at base + *o_at
  const float* lse;  // [rows]; -inf: no key, o is not read
};

// Merges the results of the cluster's n CTAs, after they have written theirs:
// threads kMergeFrom and up of each CTA call this, the others, which have given
// registers away, cluster_merge_wait().  CTA k writes dims [512 / n k, 512 / n
// (k + 1)) of the rows.  weights: n * (rows + 1) words of this CTA's shared memory.
constexpr int kMergeFrom = 128;
__device__ __forceinline__ void cluster_merge_wait() {
  cluster_sync_all();
  __syncthreads();
  cluster_sync_all();
}
__device__ __forceinline__ void cluster_merge(int n, const ClusterSide& side, float* weights, int rows,
                                              __nv_bfloat16* out, float* lse_out) {
  const float* lse = side.lse;
  const int tid = threadIdx.x - kMergeFrom, threads = blockDim.x - kMergeFrom;
  const int rank = static_cast<int>(cluster_ctarank());
  cluster_sync_all();
  for (int r = tid; r < rows; r += threads) {
    float l[kMaxCluster];
    float mx = -__builtin_huge_valf();
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) {
      l[k] = k < n ? ld_cluster_f32(mapa_shared(smem_u32(lse + r), k)) : -__builtin_huge_valf();
      mx = max_nan(mx, l[k]);
    }
    float total = mx;
    if (mx != -__builtin_huge_valf()) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) sum += exp2f(l[k] - mx);
      total = mx + log2f(sum);
    }
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k)
      if (k < n) weights[k * rows + r] = l[k] == -__builtin_huge_valf() ? 0.f : exp2f(l[k] - total);
    if (rank == 0) lse_out[r] = total;
  }
  uint32_t* places = reinterpret_cast<uint32_t*>(weights + n * rows);
  if (tid < n) places[tid] = mapa_shared(smem_u32(side.base), tid) + ld_cluster_u32(mapa_shared(smem_u32(side.o_at), tid));
  __syncthreads();
  const int per = kDv / 4 / n;  // groups of four dims of this CTA
  for (int i = tid; i < rows * per; i += threads) {
    const int r = i / per, d = 4 * (rank * per + i % per);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < n; k0 += 4) {
      float4 x[4];
      float w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w[k] = k0 + k < n ? weights[(k0 + k) * rows + r] : 0.f;
        if (w[k] != 0.f) x[k] = ld_cluster_v4(places[k0 + k] + 4 * (r * kDv + d));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (w[k] != 0.f) {
          a.x += w[k] * x[k].x;
          a.y += w[k] * x[k].y;
          a.z += w[k] * x[k].z;
          a.w += w[k] * x[k].w;
        }
    }
    *reinterpret_cast<uint2*>(out + static_cast<int64_t>(r) * kDv + d) =
        make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  }
  cluster_sync_all();  // the others may still be reading this CTA's results
}

}  // namespace mla
