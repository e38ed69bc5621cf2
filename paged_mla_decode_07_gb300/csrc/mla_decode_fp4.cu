// K12 — windowed decode over FP4 rows (mla_fp4.cuh) on tcgen05 with 8-bit operands.
//
// A key's latent values are E2M1 codes times powers of two, and so E5M2
// numbers: the rows become 8-bit operands exactly, at half the shared memory
// and half the tensor time of bf16 ones.  The other operands are split into
// 8-bit terms:
//   q (bf16, 8 significant bits), times a power of two that puts the row's
//     largest value into [128, 256): hi = E4M3(q), lo = E4M3(q - hi).  Exact for
//     values down to 2^-9 of that largest one, off by 2^-18 of it below.
//   P (fp32): three E5M2 terms of P * 2^12, each of what the last one left:
//     relative 2^-9 (what rounding to bf16 gives) down to P = 2^-23, and the
//     32 binades of E5M2 keep the weights of keys far below the largest one.
// The terms stand beside each other as columns of one MMA (N = 32 and 48 for 16
// rows, where N up to 64 costs the same time as 16) and are added in fp32 after it.
//
//   S^T [128 tokens, hi 16 | lo 16] = K [128, 512] Q^T     16 MMAs, K = 32
//   S^T [128 tokens, hi 16]        += K_rope Q_rope^T      4 bf16 MMAs, K = 16
//   O^T [128 dims, 48] x 4         += V^T P^T              16 MMAs, K = 32 tokens
// with V = the same tile, read MN-major.
//
// One CTA has 16 query rows and 256 threads, which all do the same: convert the
// tile whose codes wait in their registers into shared memory and issue the
// loads of the next one; S; softmax; O.  Two CTAs share an SM, so that one
// converts while the other's products run, and each has a whole tile (51 KB) in
// flight: neither warp roles nor more buffers.  A tile is 128 keys, two pages
// of the walk over sinks and window.
//
// Every wait is bounded (watchdog); after one that ran out all threads of the
// CTA leave together, with its products drained and its tensor memory freed.
#include "mla_cluster.cuh"
#include "mla_device.cuh"
#include "mla_fp4.cuh"
#include "mla_internal.h"
#include "mla_schedule.cuh"

namespace mla {
namespace {

constexpr int kRows = 16;      // query rows of a CTA
constexpr int kTile = 128;     // keys of a tile
constexpr int kThreads = 256;  // warps w and w + 4 share the tokens 32 (w % 4) ..; rows 8 (w / 4) ..
constexpr int kPerTok = kThreads / 16, kToks = kTile / kPerTok;  // 16 threads a token; 8 tokens a thread
constexpr int kChunkBytes = kTile * 128;                         // 128 dims of all keys
constexpr int kRopeOff = 4 * kChunkBytes;
constexpr int kQOff = kRopeOff + kChunkBytes;        // hi rows, lo rows: 4 chunks of [32][128]
constexpr int kQChunk = 2 * kRows * 128;
constexpr int kQRopeOff = kQOff + 4 * kQChunk;       // bf16 [16][64]
constexpr int kPOff = kQRopeOff + kRows * 128;       // [48][128 tokens]
constexpr int kAuxOff = kPOff + 3 * kRows * 128;
// aux: row maxima or sums of the four token groups [2][4][8], score factors [16], lse [16], barriers
constexpr int kRedOff = kAuxOff;
constexpr int kFactorOff = kRedOff + 2 * 4 * 8 * 4;
constexpr int kLseOff = kFactorOff + kRows * 4;
constexpr int kInvOff = kLseOff + kRows * 4;
constexpr int kWeightsOff = kInvOff + kRows * 4;  // cluster merge
constexpr int kMiscOff = kWeightsOff + kMaxCluster * (kRows + 1) * 4;  // abort flag, TMEM base, offset of O (0)
constexpr int kBarOff = kMiscOff + 16;
constexpr int kSmemBytes = kBarOff + 2 * 8 + 1024;  // + alignment slack
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs on an SM");
static_assert(kBarOff % 8 == 0 && kAuxOff % 16 == 0, "alignment");
constexpr uint32_t kTmemCols = 256, kSCol = 0, kOCol = 64;
constexpr float kPScale = 4096.f;  // P <= 2^kRescale goes into its terms times this, 2^15 at most
constexpr float kRescale = 3.f;    // log2 units that a score may pass the reference by before it is raised
constexpr float kNegInf = -__builtin_huge_valf();

// kind::f8f6f4, fp32 accumulation; formats 0 E4M3, 1 E5M2
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int a_format, int b_format, int a_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(a_format) << 7) | (static_cast<uint32_t>(b_format) << 10) |
         (static_cast<uint32_t>(a_mn_major) << 15) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void umma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// An E5M2 number is the upper byte of the fp16 number of its value.
__device__ __forceinline__ uint32_t e5m2x2_to_f16x2(uint32_t codes) { return __byte_perm(codes, 0, 0x1404); }
__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Reduces eight values per lane over the warp; lane l ends with value
// ((l >> 4) & 1) * 4 + ((l >> 3) & 1) * 2 + ((l >> 2) & 1).
template <class Op>
__device__ __forceinline__ float reduce8(const float (&x)[8], int lane, Op op) {
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 16;
    a[i] = op(up ? x[4 + i] : x[i], __shfl_xor_sync(0xffffffffu, up ? x[i] : x[4 + i], 16));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 8;
    b[i] = op(up ? a[2 + i] : a[i], __shfl_xor_sync(0xffffffffu, up ? a[i] : a[2 + i], 8));
  }
  const bool up = lane & 4;
  float c = op(up ? b[1] : b[0], __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 4));
  c = op(c, __shfl_xor_sync(0xffffffffu, c, 2));
  return op(c, __shfl_xor_sync(0xffffffffu, c, 1));
}

// What a thread holds of a tile on its way from global memory: 16 bytes of
// codes and a scale byte of eight tokens, 16 bytes of RoPE values of four.
struct Staged {
  uint4 code[kToks];
  uint32_t scale[kToks];
  uint4 rope[kToks / 2];
};

struct Element {
  const int32_t* table;
  int prob, L;
  KeyWalk walk;
};

// Page ids of pages j and j + 1 of the walk; those past `end` (no page of this
// CTA) are -1.
__device__ __forceinline__ int2 page_ids(const DecodeParams& p, const Element& e, int j, int end) {
  int id[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int lp = j + i < end ? e.walk.page(j + i) : -1;
    id[i] = lp >= 0 && lp < p.block_table_stride ? __ldg(e.table + lp) : -1;
  }
  return make_int2(id[0], id[1]);
}

// Whether some row sees key t, and whether every row sees all keys of a page.
__device__ __forceinline__ bool key_seen(const DecodeParams& p, int t, int L) {
  return t < L && key_in_walk(t, L, p.s_q, p.window, p.sinks);
}
__device__ __forceinline__ bool page_whole(const DecodeParams& p, int page, int L) {
  const int first = page * kPageSize, last = first + kPageSize - 1;
  if (last > L - p.s_q) return false;  // the first query token sees keys up to L - s_q
  return last < p.sinks || first > L - 1 - p.window;
}
__device__ __forceinline__ bool page_all_used(const DecodeParams& p, int page, int L) {
  const int first = page * kPageSize, last = first + kPageSize - 1;
  return last < L && (last < p.sinks || first > L - p.s_q - p.window || p.sinks > L - p.s_q - p.window);
}

// Issue the loads of pages j, j + 1 (page ids `id`).  Tokens that no row sees
// are zeros, whatever their rows hold.
__device__ __forceinline__ void stage(const DecodeParams& p, const Element& e, int j, int end, int2 id, Staged& s) {
  const int c = threadIdx.x & 15, t0 = threadIdx.x >> 4;
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int pg = h ? id.y : id.x;
    const bool real = j + h < end && pg >= 0 && pg < p.num_pages;
    const int lp = j + h < end ? e.walk.page(j + h) : 0;
    const bool all = real && page_all_used(p, lp, e.L);
    const uint8_t* base = p.kv_fp8 + static_cast<int64_t>(real ? pg : 0) * (kPageSize * kFp4RowBytes);
#pragma unroll
    for (int i = 0; i < kToks / 2; ++i) {
      const int t = t0 + kPerTok * i;
      const bool ok = all || (real && key_seen(p, lp * kPageSize + t, e.L));
      const uint8_t* row = base + t * kFp4RowBytes;
      s.code[4 * h + i] = ok ? ld_global_nc_v4(row + 16 * c) : zero;
      s.scale[4 * h + i] = ok ? __ldg(row + kFp4ScaleOffset + c) : 0u;
    }
    // RoPE: eight threads a token
#pragma unroll
    for (int i = 0; i < kToks / 4; ++i) {
      const int t = (threadIdx.x >> 3) + 32 * i;
      const bool ok = all || (real && key_seen(p, lp * kPageSize + t, e.L));
      s.rope[2 * h + i] = ok ? ld_global_nc_v4(base + t * kFp4RowBytes + kFp4RopeOffset + 16 * (threadIdx.x & 7)) : zero;
    }
  }
}

// Codes to E5M2 values in the 128-byte swizzle: block c of a token is the 16-byte
// units 2 (c % 4), 2 (c % 4) + 1 of its row of chunk c / 4.  Threads of odd chunks
// store their second unit first, so that eight of them touch all banks.
__device__ __forceinline__ void convert(const Staged& s, uint32_t smem) {
  const int c = threadIdx.x & 15, t0 = threadIdx.x >> 4;
  const uint32_t chunk = smem + (c >> 2) * kChunkBytes;
  const int u0 = 2 * (c & 3) + ((c >> 2) & 1);
#pragma unroll
  for (int i = 0; i < kToks; ++i) {
    const int t = t0 + kPerTok * i;
    const uint2 lut = fp4_lut(fp4_scale_index(s.scale[i]));
    const uint2 a = fp4_e5m2(s.code[i].x, lut), b = fp4_e5m2(s.code[i].y, lut);
    const uint2 d = fp4_e5m2(s.code[i].z, lut), f = fp4_e5m2(s.code[i].w, lut);
    const uint32_t row = chunk + t * 128;
    const bool odd = (c >> 2) & 1;
    st_shared_v4(row + ((u0 ^ (t & 7)) << 4), odd ? d.x : a.x, odd ? d.y : a.y, odd ? f.x : b.x, odd ? f.y : b.y);
    st_shared_v4(row + (((u0 ^ 1) ^ (t & 7)) << 4), odd ? a.x : d.x, odd ? a.y : d.y, odd ? b.x : f.x, odd ? b.y : f.y);
  }
#pragma unroll
  for (int i = 0; i < kToks / 2; ++i) {
    const int t = (threadIdx.x >> 3) + 32 * i;
    st_shared_v4(smem + kRopeOff + t * 128 + (((threadIdx.x & 7) ^ (t & 7)) << 4), s.rope[i].x, s.rope[i].y, s.rope[i].z,
                 s.rope[i].w);
  }
}

// The 16 query rows: hi and lo terms, RoPE values, and what a score is to be
// multiplied by.  16 threads a row, 32 latent and 4 RoPE dims each.
__device__ __forceinline__ void load_queries(const __nv_bfloat16* q, const DecodeParams& p, int prob, int g, uint8_t* smem) {
  const int r = threadIdx.x >> 4, c = threadIdx.x & 15, row = g * kRows + r;
  const bool real = row < p.rows;
  const uint4* src = reinterpret_cast<const uint4*>(q + (static_cast<int64_t>(prob) * p.rows + (real ? row : 0)) * kDqk);
  uint32_t w[16];
  uint2 rope = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = real ? __ldg(src + 4 * c + i) : make_uint4(0, 0, 0, 0);
    w[4 * i] = v.x;
    w[4 * i + 1] = v.y;
    w[4 * i + 2] = v.z;
    w[4 * i + 3] = v.w;
  }
  if (real) rope = __ldg(reinterpret_cast<const uint2*>(src + 64) + c);
  auto lo_of = [](uint32_t x) { return __uint_as_float(x << 16); };
  auto hi_of = [](uint32_t x) { return __uint_as_float(x & 0xffff0000u); };
  float amax = max_nan(max_nan(fabsf(lo_of(rope.x)), fabsf(hi_of(rope.x))), max_nan(fabsf(lo_of(rope.y)), fabsf(hi_of(rope.y))));
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = max_nan(amax, max_nan(fabsf(lo_of(w[i])), fabsf(hi_of(w[i]))));
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  // 2^k: the largest value to [128, 256), k within what a float's exponent holds both ways
  const int k = amax > 0.f ? min(max(134 - static_cast<int>(__float_as_uint(amax) >> 23), -120), 120) : 0;
  const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
  const uint32_t base = smem_u32(smem) + kQOff + (c >> 2) * kQChunk;
#pragma unroll
  for (int u = 0; u < 2; ++u) {  // 16 dims each
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[2], l[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint32_t x = w[8 * u + 2 * i + n];
        const float x0 = lo_of(x) * up, x1 = hi_of(x) * up;
        h[n] = e4m3x2(x0, x1);
        const uint32_t f = e4m3x2_to_f16x2(static_cast<uint16_t>(h[n]));
        l[n] = e4m3x2(x0 - f16x2_half_to_f32(f, 0), x1 - f16x2_half_to_f32(f, 1));
      }
      hi[i] = h[0] | (h[1] << 16);
      lo[i] = l[0] | (l[1] << 16);
    }
    const uint32_t at = base + r * 128 + (((2 * (c & 3) + u) ^ (r & 7)) << 4);
    st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
    st_shared_v4(at + kRows * 128, lo[0], lo[1], lo[2], lo[3]);
  }
  const uint32_t at = smem_u32(smem) + kQRopeOff + r * 128 + (((c >> 1) ^ (r & 7)) << 4) + 8 * (c & 1);
  st_shared_u32(at, pack_bf16x2(lo_of(rope.x) * up, hi_of(rope.x) * up));
  st_shared_u32(at + 4, pack_bf16x2(lo_of(rope.y) * up, hi_of(rope.y) * up));
  if (c == 0)  // (a row that is not finite has results that are not)
    reinterpret_cast<float*>(smem + kFactorOff)[r] =
        amax < __builtin_huge_valf() ? p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - k) << 23) : __uint_as_float(0x7fffffffu);
}

__global__ void __launch_bounds__(kThreads, 2) fp4_decode_kernel(const __nv_bfloat16* __restrict__ q, const DecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quarter = warp & 3, half = warp >> 2;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kMiscOff);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kMiscOff + 4);
  uint64_t* bar_s = reinterpret_cast<uint64_t*>(smem + kBarOff);
  uint64_t* bar_o = bar_s + 1;
  // (clusters: `part` is the problem)
  const int unit = p.cluster > 0 ? blockIdx.x / p.cluster : blockIdx.x;
  const int part = unit / p.row_groups, g = unit % p.row_groups;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const PartRecord rec = p.cluster > 0 ? cluster_share(p, part) : inline_schedule(p, part, kTile, smem, g == 0);
  // (the schedule's scratch may reach over everything below)
  if (tid == 0) {
    mbar_init(bar_s, 1);
    mbar_init(bar_o, 1);
    *abort_flag = 0;
    *reinterpret_cast<volatile int*>(smem + kMiscOff + 8) = 0;
    fence_barrier_init();
  }
  // (clusters: of a CTA without pages, or one that a wait ran out in)
  if (tid >= 32 && tid < 32 + kRows) reinterpret_cast<float*>(smem + kLseOff)[tid - 32] = kNegInf;
  if (warp == 1) {
    tmem_alloc(const_cast<uint32_t*>(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot, taddr = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
  const Watchdog wd{abort_flag, p.status, p.timeout_ns};
  const uint32_t sm = smem_u32(smem), dsm = desc_addr(smem);
  if (p.debug_stall) mbar_wait(bar_o, 0, wd);  // watchdog test: nothing completes this

  int tiles = 0;          // tiles whose scores are done: phase of both barriers
  int issued_s = 0, issued_o = 0;
  bool failed = __syncthreads_or(*abort_flag);
  const int last = rec.p1 < p.num_problems ? rec.p1 : p.num_problems - 1;
#pragma unroll 1
  for (int prob = rec.p0; prob <= last && !failed; ++prob) {
    Element e;
    e.prob = prob;
    e.L = p.cache_seqlens[prob];
    e.table = p.block_table + static_cast<int64_t>(prob) * p.block_table_stride;
    e.walk = key_walk(e.L, p.s_q, p.window, p.sinks, p.block_table_stride);
    // this CTA's pages
    const int unit_pages = p.cluster > 0 ? 1 : 2;
    const int pb = prob == rec.p0 ? unit_pages * rec.t0 : 0;
    const int pe = prob == rec.p1 ? min(unit_pages * rec.t1, e.walk.pages) : e.walk.pages;
    if (pb >= pe) continue;

    int2 id = page_ids(p, e, pb, pe);
    load_queries(q, p, prob, g, smem);
    Staged st;
    stage(p, e, pb, pe, id, st);
    int2 id_next = page_ids(p, e, pb + 2, pe);
    float ref[8], l[8], f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ref[i] = kNegInf;
      l[i] = 0.f;
    }

#pragma unroll 1
    for (int j = pb; j < pe; j += 2, ++tiles) {
      bool ok = j == pb || mbar_wait(bar_o, (tiles - 1) & 1, wd);
      if (tid < 2 && j + tid < pe) {
        const int pg = tid ? id.y : id.x;
        if (pg < 0 || pg >= p.num_pages) atomicOr(p.status, MLA_DEVICE_BAD_PAGE);
      }
      convert(st, sm);
      const int2 id_now = id;
      id = id_next;
      if (j + 2 < pe) {
        stage(p, e, j + 2, pe, id, st);
        id_next = page_ids(p, e, j + 4, pe);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      failed = __syncthreads_or(!ok);
      if (failed) break;
      ++issued_s;
      if (warp == 0) {
        tc_fence_after();
        if (elect_one()) {
          constexpr uint64_t kHi = smem_desc_hi(16, 1024);
          const uint64_t a = kHi | (dsm >> 4), b = kHi | ((dsm + kQOff) >> 4);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f8_ss(tmem + kSCol, a + ((c * kChunkBytes + 32 * k) >> 4), b + ((c * kQChunk + 32 * k) >> 4),
                         idesc_f8(kTile, 2 * kRows, 1, 0, 0), c + k > 0);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16_ss_fast(tmem + kSCol, a + ((kRopeOff + 32 * k) >> 4),
                              kHi | ((dsm + kQRopeOff + 32 * k) >> 4), idesc_bf16_f32(kTile, kRows, 0, 0), 1);
          umma_commit(bar_s);
        }
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = reinterpret_cast<const float*>(smem + kFactorOff)[8 * half + i];
      ok = mbar_wait(bar_s, tiles & 1, wd);
      tc_fence_after();

      // scores of key `lp * 64 + (lane's place)` for rows 8 half .. 8 half + 7
      float x[8];
      {
        float lo[8];
        tmem_ld_x8(taddr + kSCol + 8 * half, x);
        tmem_ld_x8(taddr + kSCol + kRows + 8 * half, lo);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (x[i] + lo[i]) * f[i];
      }
      const int jp = j + (quarter >> 1), pg = quarter >> 1 ? id_now.y : id_now.x;
      const bool real = jp < pe && pg >= 0 && pg < p.num_pages;
      const int lp = real ? e.walk.page(jp) : 0;
      if (!real || !page_whole(p, lp, e.L)) {
        const int t = lp * kPageSize + 32 * (quarter & 1) + lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int at = e.L - p.s_q + (g * kRows + 8 * half + i) / p.h_q;  // position of the row's query token
          if (!real || t > at || t >= e.L || (t >= p.sinks && t <= at - p.window)) x[i] = kNegInf;
        }
      }
      float* red = reinterpret_cast<float*>(smem + kRedOff) + 32 * half;
      {
        const float mx = reduce8(x, lane, max_nan);
        if ((lane & 3) == 0) red[8 * quarter + (lane >> 2)] = mx;
      }
      named_bar_sync(1 + half, 128);
      float mx[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        mx[i] = max_nan(max_nan(red[i], red[8 + i]), max_nan(red[16 + i], red[24 + i]));
      // raise the references that scores pass by more than kRescale (all the threads of a half alike)
      bool raise = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) raise |= !(mx[i] <= ref[i] + kRescale);
      if (raise) {
        float alpha[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          alpha[i] = 1.f;
          if (!(mx[i] <= ref[i] + kRescale)) {
            alpha[i] = ref[i] == kNegInf ? 0.f : fast_exp2(ref[i] - mx[i]);
            ref[i] = mx[i];
          }
          l[i] *= alpha[i];
        }
        if (j > pb) {
#pragma unroll 1
          for (int b = 0; b < 12; ++b) {
            const uint32_t col = taddr + kOCol + kRows * b + 8 * half;
            float o[8];
            tmem_ld_x8(col, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] *= alpha[i];
            asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(col),
                         "r"(__float_as_uint(o[0])), "r"(__float_as_uint(o[1])), "r"(__float_as_uint(o[2])),
                         "r"(__float_as_uint(o[3])), "r"(__float_as_uint(o[4])), "r"(__float_as_uint(o[5])),
                         "r"(__float_as_uint(o[6])), "r"(__float_as_uint(o[7]))
                         : "memory");
          }
          tmem_st_wait();
        }
      }
      const uint32_t pt = sm + kPOff + 8 * half * 128 + (lane & 15);
      const int pu = 2 * quarter + (lane >> 4);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        float v[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float pr = fast_exp2(x[i + n] - (ref[i + n] == kNegInf ? 0.f : ref[i + n]));
          l[i + n] += pr;
          v[n] = pr * kPScale;
        }
#pragma unroll
        for (int term = 0; term < 3; ++term) {
          const uint32_t code = e5m2x2(v[0], v[1]);
          const uint32_t at = pt + term * kRows * 128;
          st_shared_u8(at + i * 128 + ((pu ^ i) << 4), code & 0xffu);
          st_shared_u8(at + (i + 1) * 128 + ((pu ^ (i + 1)) << 4), code >> 8);
          if (term < 2) {
            const uint32_t h2 = e5m2x2_to_f16x2(code);
            v[0] -= f16x2_half_to_f32(h2, 0);
            v[1] -= f16x2_half_to_f32(h2, 1);
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      failed = __syncthreads_or(!ok);
      if (failed) break;
      ++issued_o;
      if (warp == 0) {
        tc_fence_after();
        if (elect_one()) {
          const uint64_t a = smem_desc_hi(kChunkBytes, 1024) | (dsm >> 4);
          const uint64_t b = smem_desc_hi(16, 1024) | ((dsm + kPOff) >> 4);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f8_ss(tmem + kOCol + 3 * kRows * c, a + ((c * kChunkBytes + k * 32 * 128) >> 4), b + ((32 * k) >> 4),
                         idesc_f8(128, 3 * kRows, 1, 1, 1), j > pb || k > 0);
          umma_commit(bar_o);
        }
        __syncwarp();
      }
    }
    if (failed) break;

    // row sums, then the rows
    float* red = reinterpret_cast<float*>(smem + kRedOff) + 32 * half;
    {
      const float sum = reduce8(l, lane, [](float a, float b) { return a + b; });
      if ((lane & 3) == 0) red[8 * quarter + (lane >> 2)] = sum;
    }
    bool ok = mbar_wait(bar_o, (tiles - 1) & 1, wd);
    tc_fence_after();
    failed = __syncthreads_or(!ok);
    if (failed) break;
    const bool whole = pb == 0 && pe == e.walk.pages;
    const bool final_out = whole && p.cluster == 0;
    const int slot = piece_slot(whole, prob, 2 * p.num_parts, part, prob == rec.p0);
    const bool slot_ok = final_out || p.cluster > 0 || (slot >= 0 && slot < p.max_slots);
    if (!slot_ok && tid == 0) atomicOr(p.status, MLA_DEVICE_BAD_SCHEDULE);
    float inv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float sum = red[i] + red[8 + i] + red[16 + i] + red[24 + i];
      inv[i] = sum == 0.f ? 0.f : 1.f / (sum * kPScale);
      const int r = 8 * half + i, row = g * kRows + r;
      if (quarter == 0 && lane == i && row < p.rows) {
        const float z = sum == 0.f ? kNegInf : ref[i] + log2f(sum);
        if (p.cluster > 0)
          reinterpret_cast<float*>(smem + kLseOff)[r] = z;
        else if (final_out)
          p.lse[static_cast<int64_t>(prob) * p.rows + row] = z;
        else if (slot_ok)
          p.lse_accum[static_cast<int64_t>(slot) * p.rows + row] = z;
      }
    }
    const int64_t first_row = static_cast<int64_t>(final_out ? prob : slot) * p.rows + g * kRows + 8 * half;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      float o[8], a[8], b[8];
      const uint32_t col = taddr + kOCol + 3 * kRows * c + 8 * half;
      tmem_ld_x8(col, o);
      tmem_ld_x8(col + kRows, a);
      tmem_ld_x8(col + 2 * kRows, b);
      tmem_ld_wait();
      const int d = 128 * c + 32 * quarter + lane;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = (o[i] + (a[i] + b[i])) * inv[i];
        if (p.cluster > 0) {
          reinterpret_cast<float*>(smem)[(8 * half + i) * kDv + d] = y;
        } else if (slot_ok && g * kRows + 8 * half + i < p.rows) {
          if (final_out)
            static_cast<__nv_bfloat16*>(p.out)[(first_row + i) * kDv + d] = __float2bfloat16_rn(y);
          else
            p.o_accum[(first_row + i) * kDv + d] = y;
        }
      }
    }
    tc_fence_before();
    __syncthreads();  // the next segment's first products overwrite O, its queries and sums theirs
    tc_fence_after();
  }

  if (failed) {  // products still running end (or the wait does) before the memory they use is freed
    const uint64_t t0 = global_timer_ns();
    while ((issued_s > 0 && !mbar_try_wait(bar_s, (issued_s - 1) & 1)) ||
           (issued_o > 0 && !mbar_try_wait(bar_o, (issued_o - 1) & 1)))
      if (global_timer_ns() - t0 > wd.limit_ns) break;
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  if (p.cluster > 0) {
    if (tid < kMergeFrom) {
      cluster_merge_wait();
    } else {
      const int64_t row = static_cast<int64_t>(part) * p.rows + g * kRows;
      cluster_merge(p.cluster,
                    ClusterSide{smem, reinterpret_cast<const int*>(smem + kMiscOff + 8),
                                reinterpret_cast<const float*>(smem + kLseOff)},
                    reinterpret_cast<float*>(smem + kWeightsOff), min(kRows, p.rows - g * kRows),
                    static_cast<__nv_bfloat16*>(p.out) + row * kDv, p.lse + row);
    }
  }
}

}  // namespace

cudaError_t launch_decode_fp4(const void* q, const DecodeParams& p, cudaStream_t stream) {
  // a schedule of very many problems is made in more shared memory than the tiles take (one CTA on an SM then)
  const size_t schedule = p.cluster > 0 ? 0 : schedule_scratch(p.num_problems) + 1024;
  const size_t smem = schedule > kSmemBytes ? schedule : kSmemBytes;
  cudaError_t e = allow_dynamic_smem(fp4_decode_kernel, smem, 0);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.cluster > 0 ? p.cluster * p.num_problems : p.num_parts) * p.row_groups);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fp4_decode_kernel, static_cast<const __nv_bfloat16*>(q), p);
}

}  // namespace mla
