// The schedule of windowed and shared-prefix decode.
#pragma once

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {

// Tiles of 128 keys of shared-prefix problem i: the prefix's, then those of
// the own keys of each element that the block's rows belong to.
__device__ __forceinline__ int block_first(int i, int rows) { return static_cast<int>(i * 128ll / rows); }
__device__ __forceinline__ int block_last(int i, int rows, int total_rows) {
  const long long end = i * 128ll + 128;
  return static_cast<int>(((end < total_rows ? end : total_rows) - 1) / rows);
}
__device__ __forceinline__ int key_tiles(int L, int cols) { return (pages_of(L, cols) + 1) / 2; }
__device__ __forceinline__ int block_tiles(int i, int prefix_len, int prefix_pages, const int32_t* seqlens, int cols,
                                           int rows, int total_rows, int own_keys) {
  int n = key_tiles(prefix_len, prefix_pages);
  if (own_keys) {
    const int last = block_last(i, rows, total_rows);
#pragma unroll 8
    for (int e = block_first(i, rows); e <= last; ++e) n += key_tiles(seqlens[e], cols);
  }
  return n;
}

// Tiles of problem p (PREFIX: the kernel takes calls with a shared prefix).
template <bool PREFIX>
__device__ __forceinline__ int spec_tiles(const SchedSpec& sp, int p, int tile_tokens) {
  if (PREFIX && sp.prefix_len)
    return block_tiles(p, sp.prefix_len[0], sp.prefix_pages, sp.seqlens, sp.cols, sp.rows, sp.total_rows, sp.own_keys);
  const int per = tile_tokens / kPageSize;
  return (key_walk(sp.seqlens[p], sp.s_q, sp.window, sp.sinks, sp.cols).pages + per - 1) / per;
}

// Windowed and shared-prefix decode make their schedule in every CTA of the
// decode kernel instead of in a kernel before it, which adds 5.3 us to a chain
// of 20 (4 elements, 10 pages).  Code that runs once per launch is bound by its
// instruction fetches, barriers and dependent loads (~1.2k cycles for a scan or a
// binary search; 7.7k in all when it counted the slots of split problems as the
// schedule kernel does), so it is kept to one scan, behind which the thread whose
// problems hold an end of the part finds it: a CTA needs its own part's ends, and
// the slots of partial results are named by part.
//
// The cut: problem i is a start-up cost and tiles of tile_cost each, parts are
// equal shares of all costs, as in mla_sched.cu.  A share smaller than a
// start-up and a tile would leave parts empty; then (small calls) the tiles
// alone are shared out, one or more to each part.  So every part between a
// problem's first and last holds a piece of it.
//
// Slots: a part touches at most two problems that it does not hold whole, its
// first (slot 2 k) and its last (2 k + 1).  Behind them, where problems held
// whole write partial results too, one per problem.  spans[2 i] is the slot of
// problem i's first piece and spans[2 i + 1] the part of its last one, written
// by the parts that hold its first and its last tile; the pieces between have
// slots 2 k.  A problem without tiles lies in the range of some part (those
// before the first one with tiles: of part 0), which writes (0, -1).
struct PartRecord {
  int p0, t0, p1, t1;
};

// Shared memory for a schedule of np problems.
__host__ __device__ constexpr size_t schedule_scratch(int np) { return (static_cast<size_t>(np) + 1 + 64) * 8; }

// All threads of the block; scratch: schedule_scratch() bytes of shared
// memory, 8-byte aligned, that the async proxy may write again after this
// returns.  `publish` makes this CTA write its part's spans.
template <bool PREFIX = true>
__device__ __forceinline__ PartRecord inline_schedule(const DecodeParams& p, int part, int tile_tokens,
                                                      unsigned char* scratch, bool publish) {
  const int np = p.num_problems, parts = p.num_parts, tid = threadIdx.x;
  const int lane = tid & 31, w = tid >> 5, warps = blockDim.x >> 5;
  // tiles (high word) and problems with tiles (low word), of each problem and of each warp's
  long long* held = reinterpret_cast<long long*>(scratch);  // [np], read by the thread that wrote it
  long long* warp_tot = held + np + 1;                      // [warps <= 32]
  int* const found = reinterpret_cast<int*>(warp_tot + 32);  // [2][2]
  SchedSpec spec = {};
  spec.seqlens = p.cache_seqlens;
  spec.s_q = p.s_q;
  spec.window = p.window;
  spec.sinks = p.sinks;
  spec.cols = p.block_table_stride;
  spec.prefix_len = p.prefix_len;
  spec.prefix_pages = p.prefix_pages;
  spec.rows = p.rows;
  spec.total_rows = p.total_rows;
  spec.own_keys = p.own_keys;
  auto both = [&](int i) -> long long {
    const int n = spec_tiles<PREFIX>(spec, i, tile_tokens);
    return n > 0 ? (static_cast<long long>(n) << 32) | 1 : 0;
  };
  // each thread's run of problems, then the scan over threads
  const int per = (np + blockDim.x - 1) / blockDim.x, b0 = min(tid * per, np), b1 = min(b0 + per, np);
  long long mine = 0;
#pragma unroll 1
  for (int i = b0; i < b1; ++i) {
    const long long v = both(i);
    held[i] = v;
    mine += v;
  }
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_tot[w] = x;
  __syncthreads();
  long long t = lane < warps ? warp_tot[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t += y;
  }
  const long long total = __shfl_sync(0xffffffffu, t, 31);
  x -= mine;
  if (w > 0) x += __shfl_sync(0xffffffffu, t, w - 1);
  // (x: those before this thread's run)

  // shares in costs, or in tiles
  long long tile_cost = p.tile_cost, overhead = p.overhead;
  auto cost_of = [&](long long v) { return (v >> 32) * tile_cost + (v & 0xffffffff) * overhead; };
  if (cost_of(total) < parts * (tile_cost + overhead)) {
    tile_cost = 1;
    overhead = 0;
  }
  const long long all = cost_of(total);
  const bool small = all < (1ll << 31);  // 32-bit divisions
  const long long starts = cost_of(x), ends = cost_of(x + mine);
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    const int k = part + e;
    long long at;  // floor(all * k / parts), or the k-th tile
    if (all < parts) {
      at = min(static_cast<long long>(k), all);
    } else if (small) {
      const unsigned each = static_cast<unsigned>(all) / parts, rest = static_cast<unsigned>(all) % parts;
      at = static_cast<long long>(each) * k + rest * static_cast<unsigned>(k) / parts;
    } else {
      at = all / parts * k + all % parts * k / parts;
    }
    if (at >= all) {
      if (tid == 0) {
        found[2 * e] = np;
        found[2 * e + 1] = 0;
      }
    } else if (starts <= at && at < ends) {  // one thread's run holds it
      int i = b0;
      long long before = x;
#pragma unroll 1
      for (; i + 1 < b1 && cost_of(before + held[i]) <= at; ++i) before += held[i];
      const long long o = at - cost_of(before) - overhead;
      found[2 * e] = i;
      found[2 * e + 1] = o <= 0 ? 0
                         : small ? static_cast<int>(static_cast<unsigned>(o) / static_cast<unsigned>(tile_cost))
                                 : static_cast<int>(o / tile_cost);
    }
  }
  __syncthreads();
  const PartRecord r{found[0], found[1], found[2], found[3]};
  if (publish) {
    const int first = part == 0 ? 0 : r.p0, end = r.p1 < np ? r.p1 : np - 1;
#pragma unroll 1
    for (int i = max(b0, first); i < min(b1, end + 1); ++i) {
      const int n = static_cast<int>(held[i] >> 32);
      if (n == 0) {
        p.spans[2 * i] = 0;
        p.spans[2 * i + 1] = -1;
        continue;
      }
      const int tb = i == r.p0 ? r.t0 : 0, te = i == r.p1 ? r.t1 : n;
      if (tb >= te) continue;
      if (tb == 0) p.spans[2 * i] = 2 * part + (i == r.p0 ? 0 : 1);
      if (te == n) p.spans[2 * i + 1] = part;
    }
  }
  // the scratch is free for bulk copies
  fence_proxy_async_smem();
  __syncthreads();
  return r;
}

// Slot of a piece of `problem` (counted within its kind) that part `part`
// holds; whole_base: the slots before those of problems held whole.
__device__ __forceinline__ int piece_slot(bool whole, int problem, int whole_base, int part, bool first_of_part) {
  return whole ? whole_base + problem : 2 * part + (first_of_part ? 0 : 1);
}

}  // namespace mla
