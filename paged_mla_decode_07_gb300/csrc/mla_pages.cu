// K6 — pages and slots of one step's new tokens ("assign pages").
//
// Request b holds old_b cached tokens and receives new_b more.  With 64-token
// pages it needs want_b = ceil((old_b + new_b) / 64) pages and has
// have_b = ceil(old_b / 64); page have_b + i of it is the free-list entry
//     free_pages[cursor + sum_{c < b} (want_c - have_c) + i],
// and new token i of it goes to position pos = old_b + i, i.e. slot
//     table[b][pos / 64] * 64 + pos % 64.
//
// Everything a block needs beyond its inputs is two prefix sums over the
// requests (new tokens, new pages).  Every block computes them for itself in
// shared memory: a few KB from L2 cost less than a second launch would, and
// with them no block reads what another one writes -- a token in a new page
// takes its page from the free list, a token in an old page from the table
// entry that this step leaves alone.  The cursor and the lengths may be
// updated in place (decode loops recorded as graphs do that); with more than
// one block they are then written by a second launch of one block, after
// every block of the first has read them.
//
// Bound by latency: a decode step's launch is one block with four dependent
// global reads.  Long prefill steps write 4 bytes per token.
#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kPagesThreads = 512;
constexpr int kTokensPerThread = 4;  // consecutive slots per thread: one search, one 16-byte store

struct Scan2 {
  long long a, b;
};

// Exclusive prefix sums of (a, b) over the block; returns the block's totals in *total.
__device__ Scan2 block_scan2(Scan2 v, Scan2* warp_tot, Scan2* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  Scan2 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ya = __shfl_up_sync(0xffffffffu, x.a, o), yb = __shfl_up_sync(0xffffffffu, x.b, o);
    if (lane >= o) {
      x.a += ya;
      x.b += yb;
    }
  }
  if (lane == 31) warp_tot[w] = x;
  __syncthreads();
  if (w == 0) {
    Scan2 t = lane < kPagesThreads / 32 ? warp_tot[lane] : Scan2{0, 0};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long ya = __shfl_up_sync(0xffffffffu, t.a, o), yb = __shfl_up_sync(0xffffffffu, t.b, o);
      if (lane >= o) {
        t.a += ya;
        t.b += yb;
      }
    }
    if (lane < kPagesThreads / 32) warp_tot[lane] = t;
  }
  __syncthreads();
  const Scan2 base = w > 0 ? warp_tot[w - 1] : Scan2{0, 0};
  *total = warp_tot[kPagesThreads / 32 - 1];
  return Scan2{base.a + x.a - v.a, base.b + x.b - v.b};
}

__device__ __forceinline__ int clamp_int(long long v) {
  return v > 0x7fffffffll ? 0x7fffffff : static_cast<int>(v);
}

// Last b in [lo, n) with pre[b] <= x (pre non-decreasing, pre[lo] <= x).
__device__ __forceinline__ int last_at_or_before(const int* pre, int lo, int n, int x) {
  int hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPagesThreads) assign_pages_kernel(const AssignPagesParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Scan2 warp_tot[kPagesThreads / 32];
  int* off = reinterpret_cast<int*>(smem);  // [batch + 1] first new token of request b
  int* pof = off + p.batch + 1;             // [batch + 1] first new page of request b
  int* old = pof + p.batch + 1;             // [batch]
  const int tid = threadIdx.x;
  const int cursor = min(max(p.free_cursor[0], 0), p.num_free);

  // prefix sums, each thread over a contiguous run of requests
  const int per = (p.batch + kPagesThreads - 1) / kPagesThreads;
  const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
  auto pages_of = [&](long long tokens) {
    const long long n = (tokens + kPageSize - 1) / kPageSize;
    return static_cast<int>(n < p.block_table_stride ? n : p.block_table_stride);
  };
  Scan2 mine{0, 0};
  for (int b = b0; b < b1; ++b) {
    const int o = max(p.cache_lengths[b], 0), n = max(p.new_tokens[b], 0);
    old[b] = o;
    off[b] = n;  // the count until the scan
    mine.a += n;
    mine.b += pages_of(static_cast<long long>(o) + n) - pages_of(o);
  }
  Scan2 total;
  Scan2 at = block_scan2(mine, warp_tot, &total);
  for (int b = b0; b < b1; ++b) {
    const int o = old[b], n = off[b];
    off[b] = clamp_int(at.a);
    pof[b] = clamp_int(at.b);
    at.a += n;
    at.b += pages_of(static_cast<long long>(o) + n) - pages_of(o);
    if (blockIdx.x == 0) {
      if (p.row_offsets) p.row_offsets[b] = off[b];
      if (p.cache_seqlens) p.cache_seqlens[b] = clamp_int(static_cast<long long>(o) + n);
    }
  }
  if (tid == 0) {
    off[p.batch] = clamp_int(total.a);
    pof[p.batch] = clamp_int(total.b);
    if (blockIdx.x == 0) {
      if (p.row_offsets) p.row_offsets[p.batch] = clamp_int(total.a);
      if (p.next_cursor) p.next_cursor[0] = clamp_int(min(cursor + total.b, static_cast<long long>(p.num_free)));
    }
  }
  __syncthreads();
  if (!p.fill_table) return;

  // page `i` of request b, as the table reads after this step (-1: none)
  bool no_room = off[p.batch] > p.num_tokens, bad_page = false;
  auto page_at = [&](int b, int have, long long i) -> int {
    if (i >= p.block_table_stride) {
      no_room = true;
      return -1;
    }
    int pg;
    if (i < have) {
      pg = p.block_table[static_cast<int64_t>(b) * p.block_table_stride + i];
    } else {
      const long long f = static_cast<long long>(cursor) + pof[b] + (i - have);
      if (f >= p.num_free) {
        no_room = true;
        return -1;
      }
      pg = p.free_pages[f];
    }
    if (pg < 0 || pg >= p.num_pages) {
      bad_page = true;
      return -1;
    }
    return pg;
  };

  // new table entries, one per thread
  {
    const int pages = pof[p.batch];
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPagesThreads + tid; i < pages;
         i += static_cast<int64_t>(gridDim.x) * kPagesThreads) {
      const int b = last_at_or_before(pof, 0, p.batch, static_cast<int>(i));
      const int have = pages_of(old[b]);
      const int j = have + static_cast<int>(i) - pof[b];
      p.block_table[static_cast<int64_t>(b) * p.block_table_stride + j] = page_at(b, have, j);
    }
  }

  // slots of the new tokens, four consecutive ones per thread; entries past the last token are -1
  if (p.slot_map) {
    const int tokens = off[p.batch];
    const bool vec = (reinterpret_cast<uintptr_t>(p.slot_map) & 15) == 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kPagesThreads * kTokensPerThread;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kPagesThreads + tid) * kTokensPerThread; t0 < p.num_tokens;
         t0 += step) {
      int s[kTokensPerThread];
      int b = t0 < tokens ? last_at_or_before(off, 0, p.batch, static_cast<int>(t0)) : p.batch;
      long long have_page = -1;  // page index that `pg` belongs to
      int pg = -1, have = 0;
      if (b < p.batch) have = pages_of(old[b]);
#pragma unroll
      for (int k = 0; k < kTokensPerThread; ++k) {
        const int64_t t = t0 + k;
        if (t >= tokens) {
          s[k] = -1;
          continue;
        }
        while (t >= off[b + 1]) {  // t < off[batch]: ends
          ++b;
          have = pages_of(old[b]);
          have_page = -1;
        }
        const long long pos = static_cast<long long>(old[b]) + (t - off[b]);
        if (pos / kPageSize != have_page) {
          have_page = pos / kPageSize;
          pg = page_at(b, have, have_page);
        }
        s[k] = pg < 0 ? -1 : pg * kPageSize + static_cast<int>(pos % kPageSize);
      }
      if (vec && t0 + kTokensPerThread <= p.num_tokens) {
        *reinterpret_cast<int4*>(p.slot_map + t0) = make_int4(s[0], s[1], s[2], s[3]);
      } else {
#pragma unroll
        for (int k = 0; k < kTokensPerThread; ++k)
          if (t0 + k < p.num_tokens) p.slot_map[t0 + k] = s[k];
      }
    }
  }
  if (no_room) atomicOr(p.status, MLA_DEVICE_NO_ROOM);
  if (bad_page) atomicOr(p.status, MLA_DEVICE_BAD_PAGE);
}

}  // namespace

cudaError_t launch_assign_pages(const AssignPagesParams& p, bool in_place, int sm_count, cudaStream_t stream) {
  const size_t smem = sizeof(int) * (3 * static_cast<size_t>(p.batch) + 2);
  cudaError_t e = allow_dynamic_smem(assign_pages_kernel, smem, sizeof(Scan2) * kPagesThreads / 32);
  if (e != cudaSuccess) return e;
  // one block per 2048 slots (each thread one group of four): short steps run
  // in a single block, whose in-place updates need no second launch
  const int64_t work = (static_cast<int64_t>(p.num_tokens) + kTokensPerThread - 1) / kTokensPerThread;
  int64_t grid = (work + kPagesThreads - 1) / kPagesThreads;
  if (grid < 1) grid = 1;
  if (grid > 2 * sm_count) grid = 2 * sm_count;
  AssignPagesParams first = p;
  first.fill_table = 1;
  if (in_place && grid > 1) {
    first.cache_seqlens = nullptr;
    first.next_cursor = nullptr;
  }
  assign_pages_kernel<<<static_cast<unsigned>(grid), kPagesThreads, smem, stream>>>(first);
  e = cudaGetLastError();
  if (e != cudaSuccess || !(in_place && grid > 1)) return e;
  AssignPagesParams second = p;
  second.fill_table = 0;
  second.row_offsets = nullptr;
  second.slot_map = nullptr;
  assign_pages_kernel<<<1, kPagesThreads, smem, stream>>>(second);
  return cudaGetLastError();
}

}  // namespace mla
