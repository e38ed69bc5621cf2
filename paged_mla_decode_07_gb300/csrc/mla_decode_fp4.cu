// K12 — windowed decode over FP4 rows (mla_fp4.cuh) on tcgen05 with 8-bit operands.
//
// A key's latent values are E2M1 codes times powers of two, and so E5M2
// numbers: the rows become 8-bit operands exactly, at half the shared memory
// and half the operand traffic of bf16 ones.  The other operands are split into
// 8-bit terms:
//   q (bf16, 8 significant bits), times a power of two that puts the row's
//     largest value into [128, 256): hi = E4M3(q), lo = E4M3(16 (q - hi)).  Exact
//     for values down to 2^-13 of that largest one, off by 2^-21 of it below.
//   P (fp32): three E5M2 terms of P * 2^8, each of what the last one left, times
//     16 more (E5M2 leaves an eighth at most): off by the larger of 2^-9 of
//     itself (what rounding to bf16 gives) and 2^-33 of the row's largest.  The
//     sum l has P itself, so what the terms lost would be missing from O alone:
//     with one factor for the three weights under 2^-25 were 0 in O, 2.5 % of a
//     row that has 2^20 such keys behind one large one.
// The terms stand beside each other as columns of one MMA (N = 2 R and 3 R for R
// = 16 or 32 query rows, where N up to 64 costs the same time as 16) and are
// added in fp32 after it.
//
//   S^T [128 tokens, hi R | lo R] = K [128, 512] Q^T     16 MMAs, K = 32
//   S^T [128 tokens, hi R]       += K_rope Q_rope^T      4 bf16 MMAs, K = 16
//   O^T [128 dims, 3 R] x 4      += V^T P^T              16 MMAs, K = 32 tokens
// with V = the same tile, read MN-major.
//
// A tile is 128 keys, two pages of the walk over sinks and window.  Roles: a
// warp copies codes and scales of the pages into a ring (and brings the pages
// further on into L2), one copies the RoPE values into the tile, sixteen warps
// turn codes into the tile's E5M2 values, one issues the products of S, one those
// of O, eight have the softmax and the results.  Two tile buffers, whose chunks
// are handed on in pairs.
//
// What bounds it: not memory (64 x 16 rows over 2048 to 16384 keys take 73 us, 3.2
// TB/s, where the rows' bytes take 35) but 1.74 us for each of a CTA's 30 tiles (32
// rows: 2.7), 14 us of start, end and merge of any call, and 4.6 us for each segment
// behind a CTA's first (32 rows: 5; from calls of one, two and four equal segments a
// CTA).  A tile's time is the chain through its buffer, 3.3k cycles (32 rows: 4.5k):
// stores of the values, products of S, softmax, products of O, the next values.  In it
// the products (1540 cycles of operand reads at the 128 bytes a clock of shared memory)
// and the stores share that bandwidth, ~2800 cycles of it.  More buffers have no room (a tile of E5M2 values is 64 KB); the
// same tiles in bf16 would be twice that and twice the operand traffic.  Measured
// on the way (us, that call): all threads doing everything, two CTAs an SM, codes
// prefetched in registers, 120 (the loads' scoreboards are those of the other
// steps); roles with eight conversion warps 122, products of S and O from one warp in
// whichever order is ready 124, maxima exchanged in raised tiles alone 115, sixteen
// conversion warps, P by rows and a warp each for S and O 87, values held in
// registers until their buffer is free 83, row sums by lanes 81 (cold caches).  32
// rows (32 x 128 rows over 1001 to 8191 keys): 157, with the same steps 101, waits that
// end early first and L2 brought in behind the first pages 97 (92 in a row of calls),
// four pages ahead at once for one page six ahead 91.
// Not kept there: two pages of codes at once in runs of 32 tokens, one RoPE buffer and
// a page held as codes, which shorten the chain to 4.0k and spill (91; 128 x 16 rows of
// a window 87 for 86); in runs of 16 tokens the copies bound it (114).
// With more than 32 rows every 32 of them convert and multiply a page again: 64 x 64
// rows take 159 us, 64 x 128 rows 293, where the kernels over bf16 rows take 155 and 185.
//
// Every wait is bounded (watchdog); after one that ran out every role leaves,
// copies and products are drained and the tensor memory is freed.
#include "mla_cluster.cuh"
#include "mla_device.cuh"
#include "mla_fp4.cuh"
#include "mla_internal.h"
#include "mla_schedule.cuh"

namespace mla {
namespace {

constexpr int kTile = 128;                // keys of a tile
constexpr int kChunkBytes = kTile * 128;  // 128 dims of all keys
constexpr int kTileBytes = 4 * kChunkBytes;
constexpr int kRawRow = kFp4RopeOffset;   // codes and scales; 17 16-byte units, so rows lie on different banks
constexpr int kRawBytes = kPageSize * kRawRow;
constexpr int kConvWarps = 16, kSoftWarps = 8;
constexpr int kThreads = 32 * (4 + kConvWarps + kSoftWarps);
constexpr uint32_t kLaunchRegs = 72;
constexpr int kFactors = 4;  // segments whose score factors are kept
constexpr int kFlags = 4;    // tiles whose page states are kept
constexpr int kAhead = 4;    // pages brought into L2 ahead of their copy

template <int R>
struct Cfg {
  // setmaxnreg hands out what the block was launched with and waits for ever for more
  static constexpr uint32_t kRegsCtl = 56, kRegsConv = R == 16 ? 64 : 56, kRegsSoft = R == 16 ? 96 : 112;
  static_assert(kRegsCtl + 4 * kRegsConv + 2 * kRegsSoft <= 7 * kLaunchRegs && kThreads * kLaunchRegs <= 65536,
                "register split");
  static constexpr int kRaw = R == 16 ? 2 : 1;    // pages of the ring
  static constexpr int kPBufs = R == 16 ? 2 : 1;  // buffers of P
  static constexpr int kRows = R / 2;             // rows of a softmax thread
  static constexpr int kRopeOff = 2 * kTileBytes;
  static constexpr int kQOff = kRopeOff + 2 * kChunkBytes;  // hi rows, lo rows: 4 chunks of [2 R][128]
  static constexpr int kQChunk = 2 * R * 128;
  static constexpr int kQRopeOff = kQOff + 4 * kQChunk;  // bf16 [R][64]
  static constexpr int kPOff = kQRopeOff + R * 128;      // [3 R / 16][128 tokens][16 rows]
  static constexpr int kPBytes = 3 * R * 128;
  static constexpr int kRawOff = kPOff + kPBufs * kPBytes;
  static constexpr int kAuxOff = kRawOff + kRaw * kRawBytes;
  // aux: row maxima or sums of the four token groups [2 tiles][2][4][R / 2], score
  // factors [kFactors][R], lse [R], page states [kFlags][2] and [kRaw], abort flag,
  // TMEM base, offset of O (0), barriers
  static constexpr int kRedOff = kAuxOff;
  static constexpr int kFactorOff = kRedOff + 2 * 4 * R * 4;
  static constexpr int kLseOff = kFactorOff + kFactors * R * 4;
  static constexpr int kFlagOff = kLseOff + R * 4;
  static constexpr int kRawFlagOff = kFlagOff + kFlags * 2 * 4;
  static constexpr int kMiscOff = kRawFlagOff + 2 * 4;
  static constexpr int kBarOff = (kMiscOff + 12 + 7) / 8 * 8;
  static constexpr int kNumBars = 2 * kRaw + 2 * 3 + 4 * 2 + 1;
  // (1024 bytes of alignment; R = 32 has 16 fewer to spare and needs none: dynamic
  // shared memory without static variables starts at its multiple, which the kernel checks)
  static constexpr int kSmemBytes = kBarOff + kNumBars * 8 + (R == 16 ? 1024 : 0);
  static constexpr uint32_t kTmemCols = R == 16 ? 256 : 512;
  static constexpr uint32_t kSCol = 0, kOCol = 4 * R;
  static_assert(4 * R + 12 * R <= static_cast<int>(kTmemCols), "tensor memory");
  static_assert(kBarOff % 8 == 0 && kAuxOff % 16 == 0 && kRawOff % 128 == 0, "alignment");
  static_assert(kSmemBytes <= 232448, "shared memory");
  static_assert(schedule_scratch(kMaxProblems) <= kAuxOff, "a schedule is made where the tiles will be");
  static_assert(kMaxCluster * (R + 1) * 4 <= kPBytes, "weights of a cluster's merge, in P's place");
};
constexpr float kPLog2 = 8.f;      // P is held at 2^8 times its value, 2^15 at most
constexpr float kPStep = 16.f;     // and its second and third term at 16 times what the one before left: 2^11 of 2^15
constexpr float kQStep = 16.f;     // the second term of q is held at 16 times what the first left (8 of 256 at most)
constexpr float kRescale = 7.f;    // log2 units that a score may pass the reference by before it is raised
constexpr float kNegInf = -__builtin_huge_valf();
constexpr uint32_t kHalfBar = 1;   // named barriers of the softmax warps of a half of the rows

// kind::f8f6f4, fp32 accumulation; formats 0 E4M3, 1 E5M2
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int a_format, int b_format, int mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(a_format) << 7) | (static_cast<uint32_t>(b_format) << 10) |
         (static_cast<uint32_t>(mn_major) * (3u << 15)) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// P lies MN-major without swizzle: 128-byte blocks of 8 tokens with 16 rows
// each, those of the next tokens behind them (leading offset), those of the next
// 16 rows 2 KB on (stride offset): a thread writes its rows of a token at once.
constexpr uint32_t kDescHiP = (2048u >> 4) | (1u << 14);
// Descriptors as words: the code between two MMAs has to be short where the warp
// that issues them shares its scheduler with busy ones.
__device__ __forceinline__ void umma_f8_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                           bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %6};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(kDescHi), "r"(b_hi));
}
__device__ __forceinline__ void umma_bf16_words(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
      "setp.ne.b32 p, 1, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(kDescHi));
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
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[N]) {
  if constexpr (N == 8)
    tmem_ld_x8(taddr, v);
  else
    tmem_ld_x16(taddr, v);
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&v)[16]) { tmem_st_x16(taddr, v); }
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}

// Reduces N values per lane over the warp; lane l ends with value l / (32 / N).
template <int N, class Op>
__device__ __forceinline__ float reduce_rows(const float (&x)[N], int lane, Op op) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = x[i];
  int o = 16;
#pragma unroll
  for (int n = N / 2; n >= 1; n /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = op(up ? v[n + i] : v[i], __shfl_xor_sync(0xffffffffu, up ? v[i] : v[n + i], o));
  }
#pragma unroll
  for (; o >= 1; o /= 2) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
}

struct Bars {
  uint64_t* raw_full;   // [kRaw] codes and scales of a page have landed
  uint64_t* raw_empty;  // [kRaw] the conversion warps have read them
  uint64_t* rope_full;  // [2] RoPE values of a tile have landed
  uint64_t* k_full;     // [2][2] values of a tile's pair of chunks (and of Q, before a segment's first) are written
  uint64_t* s_full;     // [2] scores of a tile are in tensor memory
  uint64_t* p_full;     // [2] P of a tile is written (and its scores read)
  uint64_t* done;       // [2][2] the products of O of a pair are done: the pair (after the second P) is free
  uint64_t* o_free;     // O of a segment has been read
};

// What a CTA has of problem `prob`: pages pb .. pe of its walk.
struct Segment {
  const int32_t* table;
  int L, pb, pe;
  KeyWalk walk;
};
struct Range {
  PartRecord rec;
  int last;
  __device__ bool get(const DecodeParams& p, int prob, Segment& s) const {
    s.L = p.cache_seqlens[prob];
    s.table = p.block_table + static_cast<int64_t>(prob) * p.block_table_stride;
    s.walk = key_walk(s.L, p.s_q, p.window, p.sinks, p.block_table_stride);
    const int unit = p.cluster > 0 ? 1 : 2;  // (clusters share out pages, schedules tiles)
    s.pb = prob == rec.p0 ? unit * rec.t0 : 0;
    s.pe = prob == rec.p1 ? min(unit * rec.t1, s.walk.pages) : s.walk.pages;
    return s.pb < s.pe;
  }
};
// Page id of page j of the segment, -1 if it has none that is usable.
__device__ __forceinline__ int page_id(const DecodeParams& p, const Segment& s, int j) {
  if (j >= s.pe) return -1;
  const int lp = s.walk.page(j);
  const int id = lp < p.block_table_stride ? __ldg(s.table + lp) : -1;
  return id >= 0 && id < p.num_pages ? id : -1;
}

// Whether some row sees key t; whether some row sees each key of a page; whether every row sees all of them.
__device__ __forceinline__ bool key_seen(const DecodeParams& p, int t, int L) {
  return t < L && key_in_walk(t, L, p.s_q, p.window, p.sinks);
}
__device__ __forceinline__ bool page_used(const DecodeParams& p, int page, int L) {
  const int first = page * kPageSize, last = first + kPageSize - 1, past = L - p.s_q - p.window;
  return last < L && (last < p.sinks || first > past || p.sinks > past);
}
__device__ __forceinline__ bool page_whole(const DecodeParams& p, int page, int L) {
  const int first = page * kPageSize, last = first + kPageSize - 1;
  if (last > L - p.s_q) return false;  // the first query token sees keys up to L - s_q
  return last < p.sinks || first > L - 1 - p.window;
}

__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const Watchdog& wd) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, wd));
}
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, const Watchdog& wd) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > wd.limit_ns) break;
}

// ---------------------------------------------------------------------------
// copies: codes and scales (one warp), RoPE values (one warp)
// ---------------------------------------------------------------------------
template <int R>
__device__ void copy_codes(const CUtensorMap* tm, const DecodeParams& p, const Range& rg, uint8_t* smem, const Bars& bars,
                           const Watchdog& wd) {
  using C = Cfg<R>;
  const int lane = threadIdx.x & 31;
  const uint64_t pol = p.evict_first ? l2_policy_evict_first() : l2_policy_evict_normal();
  volatile int* flags = reinterpret_cast<volatile int*>(smem + C::kRawFlagOff);
  int u = 0;
#pragma unroll 1
  for (int prob = rg.rec.p0; prob <= rg.last; ++prob) {
    Segment s;
    if (!rg.get(p, prob, s)) continue;
    int ids = -1, next = page_id(p, s, s.pb + lane);  // of 32 pages from j0 on, and of the 32 behind them
    int j0 = s.pb - 32, far = 0;  // far: the first page that has not been brought into L2
#pragma unroll 1
    for (int j = s.pb; j < s.pe; ++j, ++u) {
      if (j - j0 == 32) {
        j0 = j;
        ids = next;
        next = page_id(p, s, j + 32 + lane);
      }
      const int id = __shfl_sync(0xffffffffu, ids, j - j0), slot = u % C::kRaw;
      if (u >= C::kRaw && !wait_warp(bars.raw_empty + slot, ((u / C::kRaw) - 1) & 1, wd)) goto out;
      if (lane == 0) {
        if (id < 0) atomicOr(p.status, MLA_DEVICE_BAD_PAGE);
        flags[slot] = id;
        mbar_arrive_expect_tx(bars.raw_full + slot, id < 0 ? 0 : kRawBytes);
        if (id >= 0)
          tma_load_2d(smem + C::kRawOff + slot * kRawBytes, tm, bars.raw_full + slot, 0, id * kPageSize, pol);
      }
      __syncwarp();
      // pages up to j + kAhead into L2 (64 are known from j0 on), the first ones behind the copies of a whole ring
      if (u >= C::kRaw - 1) {
        const int page = max(far, j + 1) + lane, at = page - j0;
        const int low = __shfl_sync(0xffffffffu, ids, at & 31), high = __shfl_sync(0xffffffffu, next, at & 31);
        const int ahead = at < 32 ? low : high;
        if (page <= j + kAhead && ahead >= 0)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                           p.kv_fp8 + static_cast<int64_t>(ahead) * (kPageSize * kFp4RowBytes)),
                       "r"(kPageSize * kFp4RowBytes)
                       : "memory");
        far = j + kAhead + 1;
      }
    }
  }
out:
  // no copy may be in flight when the CTA ends
  if (lane == 0)
    for (int i = u > C::kRaw ? u - C::kRaw : 0; i < u; ++i) drain(bars.raw_full + i % C::kRaw, (i / C::kRaw) & 1, wd);
  __syncwarp();
}

template <int R>
__device__ void copy_rope(const CUtensorMap* tm, const DecodeParams& p, const Range& rg, uint8_t* smem, const Bars& bars,
                          const Watchdog& wd) {
  using C = Cfg<R>;
  const int lane = threadIdx.x & 31;
  const uint64_t pol = p.evict_first ? l2_policy_evict_first() : l2_policy_evict_normal();
  int i = 0;  // tiles
#pragma unroll 1
  for (int prob = rg.rec.p0; prob <= rg.last; ++prob) {
    Segment s;
    if (!rg.get(p, prob, s)) continue;
    int id[2], next[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) next[h] = page_id(p, s, s.pb + h);
#pragma unroll 1
    for (int j = s.pb; j < s.pe; j += 2, ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        id[h] = next[h];
        next[h] = page_id(p, s, j + 2 + h);
      }
      const int b = i & 1;
      if (i >= 2 && !wait_warp(bars.s_full + b, ((i >> 1) - 1) & 1, wd)) goto out;
      if (lane == 0) {
        mbar_arrive_expect_tx(bars.rope_full + b, ((id[0] >= 0) + (id[1] >= 0)) * (kChunkBytes / 2));
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (id[h] >= 0)
            tma_load_2d(smem + C::kRopeOff + b * kChunkBytes + h * (kChunkBytes / 2), tm, bars.rope_full + b,
                        kFp4RopeOffset / 2, id[h] * kPageSize, pol);
      }
      __syncwarp();
    }
  }
out:
  if (lane == 0)
    for (int k = i > 2 ? i - 2 : 0; k < i; ++k) drain(bars.rope_full + (k & 1), (k >> 1) & 1, wd);
  __syncwarp();
}

// ---------------------------------------------------------------------------
// conversion warps
// ---------------------------------------------------------------------------
// The R query rows: hi and lo terms, RoPE values, and what a score is to be
// multiplied by.  512 / R threads a row.
template <int R>
__device__ __forceinline__ void load_queries(const __nv_bfloat16* q, const DecodeParams& p, int prob, int g, uint8_t* smem,
                                             float* factor) {
  using C = Cfg<R>;
  constexpr int kPer = 512 / R, kUnits = 32 / kPer, kRope = 32 / kPer;  // threads a row; 16 dims, RoPE pairs a thread
  const int ct = threadIdx.x - 128;
  const int r = ct / kPer, c = ct % kPer, row = g * R + r;
  const bool real = row < p.rows;
  const uint4* src = reinterpret_cast<const uint4*>(q + (static_cast<int64_t>(prob) * p.rows + (real ? row : 0)) * kDqk);
  uint32_t w[8 * kUnits], rope[kRope];
#pragma unroll
  for (int i = 0; i < 2 * kUnits; ++i) {
    const uint4 v = real ? __ldg(src + 2 * kUnits * c + i) : make_uint4(0, 0, 0, 0);
    w[4 * i] = v.x;
    w[4 * i + 1] = v.y;
    w[4 * i + 2] = v.z;
    w[4 * i + 3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < kRope; ++i) rope[i] = real ? __ldg(reinterpret_cast<const uint32_t*>(src + 64) + c * kRope + i) : 0u;
  auto lo_of = [](uint32_t x) { return __uint_as_float(x << 16); };
  auto hi_of = [](uint32_t x) { return __uint_as_float(x & 0xffff0000u); };
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kRope; ++i) amax = max_nan(amax, max_nan(fabsf(lo_of(rope[i])), fabsf(hi_of(rope[i]))));
#pragma unroll
  for (int i = 0; i < 8 * kUnits; ++i) amax = max_nan(amax, max_nan(fabsf(lo_of(w[i])), fabsf(hi_of(w[i]))));
#pragma unroll
  for (int o = kPer / 2; o >= 1; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  // 2^k: the largest value to [128, 256), k within what a float's exponent holds both ways
  const int k = amax > 0.f ? min(max(134 - static_cast<int>(__float_as_uint(amax) >> 23), -120), 120) : 0;
  const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
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
        l[n] = e4m3x2((x0 - f16x2_half_to_f32(f, 0)) * kQStep, (x1 - f16x2_half_to_f32(f, 1)) * kQStep);
      }
      hi[i] = h[0] | (h[1] << 16);
      lo[i] = l[0] | (l[1] << 16);
    }
    const int d = kUnits * c + u;  // 16-byte unit of the row's 32
    const uint32_t at = smem_u32(smem) + C::kQOff + (d >> 3) * C::kQChunk + r * 128 + (((d & 7) ^ (r & 7)) << 4);
    st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
    st_shared_v4(at + R * 128, lo[0], lo[1], lo[2], lo[3]);
  }
#pragma unroll
  for (int i = 0; i < kRope; ++i) {
    const int word = kRope * c + i;
    st_shared_u32(smem_u32(smem) + C::kQRopeOff + r * 128 + (((word >> 2) ^ (r & 7)) << 4) + 4 * (word & 3),
                  pack_bf16x2(lo_of(rope[i]) * up, hi_of(rope[i]) * up));
  }
  if (c == 0)  // (a row that is not finite has results that are not)
    factor[r] = amax < __builtin_huge_valf() ? p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - k) << 23)
                                             : __uint_as_float(0x7fffffffu);
}

// Codes to E5M2 values in the 128-byte swizzle.  The values wait in registers (16
// rows: of the whole tile) until the products that read its buffer are done, and
// are handed on two chunks at a time.  A thread has block c0 of chunk d and of chunk d + 2 of token t: the 16-byte units
// 2 c0, 2 c0 + 1 of their rows (lanes are dealt out so that the stores of eight of
// them touch all banks).  Bound by the logical and permute instructions, 64
// lanes a clock: 36 for 32 values, ~1150 cycles for a tile.
template <int R>
__device__ void convert(const __nv_bfloat16* q, const DecodeParams& p, const Range& rg, int g, uint8_t* smem, const Bars& bars,
                        const Watchdog& wd) {
  using C = Cfg<R>;
  constexpr int kHold = C::kRaw;  // pages whose values are held
  const int ct = threadIdx.x - 128;
  const int c0 = ct & 3, t = ((ct >> 2) & 3) | ((ct >> 5) << 2), d = (ct >> 4) & 1;
  const uint32_t at = smem_u32(smem) + d * kChunkBytes + t * 128;
  const uint32_t at0 = ((2 * c0) ^ (t & 7)) << 4, at1 = ((2 * c0 + 1) ^ (t & 7)) << 4;
  const volatile int* flags = reinterpret_cast<const volatile int*>(smem + C::kRawFlagOff);
  volatile int* states = reinterpret_cast<volatile int*>(smem + C::kFlagOff);
  int u = 0, i = 0, seg = 0;
#pragma unroll 1
  for (int prob = rg.rec.p0; prob <= rg.last; ++prob) {
    Segment s;
    if (!rg.get(p, prob, s)) continue;
    // the last products that read the queries of the segment before
    if (i > 0 && !wait_warp(bars.s_full + ((i - 1) & 1), ((i - 1) >> 1) & 1, wd)) return;
    load_queries<R>(q, p, prob, g, smem, reinterpret_cast<float*>(smem + C::kFactorOff) + (seg % kFactors) * R);
    ++seg;
#pragma unroll 1
    for (int j = s.pb; j < s.pe; j += 2, ++i) {
      const int b = i & 1, pages = min(2, s.pe - j);
#pragma unroll 1
      for (int h0 = 0; h0 < pages; h0 += kHold) {
      uint4 out[kHold][2][2];
#pragma unroll
      for (int n = 0; n < kHold; ++n) {
        const int h = h0 + n;
        if (h >= pages) break;
        const int slot = u % C::kRaw, lp = s.walk.page(j + h);
        if (!wait_warp(bars.raw_full + slot, (u / C::kRaw) & 1, wd)) return;
        ++u;
        const int id = flags[slot];
        const bool real = id >= 0;
        if (ct == 0) {
          states[2 * (i % kFlags) + h] = real;
          if (h == 0) states[2 * (i % kFlags) + 1] = 0;
        }
        const uint8_t* row = smem + C::kRawOff + slot * kRawBytes + t * kRawRow;
        uint4 code[2];
        uint32_t scale[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          code[k] = *reinterpret_cast<const uint4*>(row + 128 * k + 64 * d + 16 * c0);
          scale[k] = row[kFp4ScaleOffset + 8 * k + 4 * d + c0];
        }
        // The slot is handed back when the warp's reads of it are complete.  A read is
        // complete where an instruction has its result as an operand; the arrival waits
        // for no read by itself, and the copy that it lets go is no access of this proxy
        // (an arrival right behind the reads has let the next page's copy overtake them,
        // where there is one slot and pages are in L2).  So a vote, in which every lane
        // has a word of each of its reads as an operand, stands before the arrival, and a
        // branch on it holds the two in order; the branch is all that the fence in it is for.
        // (A proxy fence instead of the argument: 64 x 16 rows 73.6 -> 76.4 us, 32 x 128 91.3 -> 93.0.)
        if (__any_sync(0xffffffffu, (code[0].x ^ code[1].x) + (scale[0] ^ scale[1]) + id == 0x9e3779b9u)) __threadfence_block();
        arrive_warp(bars.raw_empty + slot);
        if (!real || !page_used(p, lp, s.L)) {
          // a token that no row sees is zeros, whatever its row holds
          if (!real || !key_seen(p, lp * kPageSize + t, s.L)) code[0] = code[1] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint2 lut = fp4_lut(fp4_scale_index(scale[k]));
          const uint2 x = fp4_e5m2(code[k].x, lut), y = fp4_e5m2(code[k].y, lut);
          const uint2 z = fp4_e5m2(code[k].z, lut), w = fp4_e5m2(code[k].w, lut);
          out[n][k][0] = make_uint4(x.x, x.y, y.x, y.y);
          out[n][k][1] = make_uint4(z.x, z.y, w.x, w.y);
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (h0 == 0 && i >= 2 && !wait_warp(bars.done + 2 * b + k, ((i >> 1) - 1) & 1, wd)) return;
#pragma unroll
        for (int n = 0; n < kHold; ++n) {
          if (h0 + n >= pages) break;
          const uint32_t to = at + b * kTileBytes + 2 * k * kChunkBytes + (h0 + n) * (kChunkBytes / 2);
          st_shared_v4(to + at0, out[n][k][0].x, out[n][k][0].y, out[n][k][0].z, out[n][k][0].w);
          st_shared_v4(to + at1, out[n][k][1].x, out[n][k][1].y, out[n][k][1].z, out[n][k][1].w);
        }
        if (h0 + kHold < pages) continue;
        fence_proxy_async_smem();
        arrive_warp(bars.k_full + 2 * b + k);
      }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// products: those of S (one warp), those of O (one warp)
// ---------------------------------------------------------------------------
template <int R>
__device__ void score_products(const DecodeParams& p, const Range& rg, uint32_t tmem, uint8_t* smem, const Bars& bars,
                               const Watchdog& wd) {
  using C = Cfg<R>;
  const uint32_t base = desc_addr(smem);
  const uint32_t qd = desc_lo(base + C::kQOff, 16), qr = desc_lo(base + C::kQRopeOff, 16);
  int i = 0;
  bool ok = true;
#pragma unroll 1
  for (int prob = rg.rec.p0; prob <= rg.last && ok; ++prob) {
    Segment s;
    if (!rg.get(p, prob, s)) continue;
#pragma unroll 1
    for (int j = s.pb; j < s.pe && ok; j += 2, ++i) {
      const int b = i & 1, ph = (i >> 1) & 1;
      const uint32_t a = desc_lo(base + b * kTileBytes, 16), ar = desc_lo(base + C::kRopeOff + b * kChunkBytes, 16);
      const uint32_t d = tmem + C::kSCol + 2 * R * b;
      // the scores of two tiles before have been read, the RoPE values are there (each wait takes
      // about a hundred cycles: those that end early come first)
      if (i >= 2) ok = wait_warp(bars.p_full + b, ph ^ 1, wd);
      ok = ok && wait_warp(bars.rope_full + b, ph, wd);
#pragma unroll
      for (int part = 0; part < 3; ++part) {  // two chunks, two chunks, RoPE
        if (part < 2) ok = ok && wait_warp(bars.k_full + 2 * b + part, ph, wd);
        tc_fence_after();
        if (elect_one()) {
          if (ok && part < 2) {
#pragma unroll
            for (int c = 2 * part; c < 2 * part + 2; ++c)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_f8_ss(d, a + ((c * kChunkBytes + 32 * k) >> 4), qd + ((c * C::kQChunk + 32 * k) >> 4), kDescHi,
                           idesc_f8(kTile, 2 * R, 1, 0, 0), c + k > 0);
          } else if (ok) {
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_bf16_words(d, ar + 2 * k, qr + 2 * k, idesc_bf16_f32(kTile, R, 0, 0));
          }
          if (part == 2) umma_commit(bars.s_full + b);  // (of what has been issued, where a wait ran out too)
        }
        __syncwarp();
      }
    }
  }
  // products still running end (or the waits do) before the memory they use is freed
  if (i > 0) drain(bars.s_full + ((i - 1) & 1), ((i - 1) >> 1) & 1, wd);
}

template <int R>
__device__ void value_products(const DecodeParams& p, const Range& rg, uint32_t tmem, uint8_t* smem, const Bars& bars,
                               const Watchdog& wd) {
  using C = Cfg<R>;
  const uint32_t base = desc_addr(smem);
  int i = 0, seg = 0;
  bool ok = true;
#pragma unroll 1
  for (int prob = rg.rec.p0; prob <= rg.last && ok; ++prob) {
    Segment s;
    if (!rg.get(p, prob, s)) continue;
    if (seg > 0) ok = wait_warp(bars.o_free, (seg - 1) & 1, wd);
    ++seg;
#pragma unroll 1
    for (int j = s.pb; j < s.pe; j += 2, ++i) {
      const int b = i & 1, steps = 2 * min(2, s.pe - j);  // (the second half of a tile of one page holds no values)
      ok = ok && wait_warp(bars.p_full + b, (i >> 1) & 1, wd);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t a = desc_lo(base + b * kTileBytes, kChunkBytes);
        const uint32_t pd = desc_lo(base + C::kPOff + (i % C::kPBufs) * C::kPBytes, 128);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < steps)
              umma_f8_ss(tmem + C::kOCol + 3 * R * c, a + ((c * kChunkBytes + k * 32 * 128) >> 4), pd + ((512 * k) >> 4), kDescHiP,
                         idesc_f8(128, 3 * R, 1, 1, 1), j > s.pb || k > 0);
          if (c & 1) umma_commit(bars.done + 2 * b + (c >> 1));
        }
      }
      __syncwarp();
    }
  }
  if (i > 0) drain(bars.done + 2 * ((i - 1) & 1) + 1, ((i - 1) >> 1) & 1, wd);
}

// ---------------------------------------------------------------------------
// softmax and results: warps w and w + 4 share the tokens 32 (w % 4) .., rows R / 2 (w / 4) ..
// ---------------------------------------------------------------------------
template <int R>
__device__ void softmax(const DecodeParams& p, const Range& rg, int g, int part, uint32_t tmem, uint8_t* smem,
                        const Bars& bars, const Watchdog& wd) {
  using C = Cfg<R>;
  constexpr int N = C::kRows;
  const int sw = (threadIdx.x >> 5) - 4 - kConvWarps, lane = threadIdx.x & 31, quarter = sw & 3, half = sw >> 2;
  const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
  const volatile int* states = reinterpret_cast<const volatile int*>(smem + C::kFlagOff);
  float* const red2 = reinterpret_cast<float*>(smem + C::kRedOff) + 4 * N * half;
  const auto add = [](float a, float b) { return a + b; };
  bool ok = true;
  if (p.debug_stall) ok = mbar_wait(bars.o_free, 0, wd);  // watchdog test: nothing completes this before this role has run
  int i = 0, seg = 0;
#pragma unroll 1
  for (int prob = rg.rec.p0; prob <= rg.last; ++prob) {
    Segment s;
    if (!rg.get(p, prob, s)) continue;
    const float* factor = reinterpret_cast<const float*>(smem + C::kFactorOff) + (seg % kFactors) * R + N * half;
    ++seg;
    float down[N], l[N], f[N];
    uint32_t seen = 0;  // rows that have a reference
#pragma unroll
    for (int r = 0; r < N; ++r) down[r] = l[r] = 0.f;
#pragma unroll 1
    for (int j = s.pb; j < s.pe; j += 2, ++i) {
      const int b = i & 1;
      // (the conversion warps' page states and factors are read below; two buffers of P: this
      // tile's is free where its scores are to come)
      ok = ok && mbar_wait(bars.k_full + 2 * b, (i >> 1) & 1, wd);
      if (C::kPBufs == 2 && i >= 2) ok = ok && mbar_wait(bars.done + 2 * b + 1, ((i >> 1) - 1) & 1, wd);
      ok = ok && mbar_wait(bars.s_full + b, (i >> 1) & 1, wd);
      tc_fence_after();
      if (j == s.pb) {
#pragma unroll
        for (int r = 0; r < N; ++r) f[r] = factor[r];
      }
      // y = score - reference + kPLog2; a row's reference is the largest score of its
      // first tile, raised where a score passes it by more than kRescale, which a
      // vote finds: the maxima are exchanged in such tiles alone.
      float y[N];
      {
        float lo[N];
        tmem_ld(taddr + C::kSCol + 2 * R * b + N * half, y);
        tmem_ld(taddr + C::kSCol + 2 * R * b + R + N * half, lo);
        tmem_ld_wait();
#pragma unroll
        for (int r = 0; r < N; ++r) y[r] = fmaf(fmaf(lo[r], 1.f / kQStep, y[r]), f[r], down[r]);
      }
      const int jp = j + (quarter >> 1);
      const bool real = states[2 * (i % kFlags) + (quarter >> 1)] != 0;
      const int lp = jp < s.pe ? s.walk.page(jp) : 0;
      if (!real || !page_whole(p, lp, s.L)) {
        const int t = lp * kPageSize + 32 * (quarter & 1) + lane;
#pragma unroll
        for (int r = 0; r < N; ++r) {
          const int at = s.L - p.s_q + (g * R + N * half + r) / p.h_q;  // position of the row's query token
          if (!real || t > at || t >= s.L || (t >= p.sinks && t <= at - p.window)) y[r] = kNegInf;
        }
      }
      float top = y[0];
#pragma unroll
      for (int r = 1; r < N; ++r) top = max_nan(top, y[r]);
      bool vote = !ok || !(top <= kRescale + kPLog2);
      if (seen != (1u << N) - 1) {
#pragma unroll
        for (int r = 0; r < N; ++r) vote |= !((seen >> r) & 1) && y[r] != kNegInf;
      }
      // (the four warps of a half act and leave alike)
      if (named_bar_or(kHalfBar + half, 128, vote)) {
        // two buffers: a warp that is ahead passes no vote of the tile behind it
        float* red = red2 + (i & 1) * 4 * R;
        const float mine = reduce_rows<N>(y, lane, max_nan);
        if (lane % (32 / N) == 0) red[N * quarter + lane / (32 / N)] = mine;
        if (!named_bar_and(kHalfBar + half, 128, ok)) return;
        float alpha[N];
#pragma unroll
        for (int r = 0; r < N; r += 4) {
          float4 m[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) m[k] = *reinterpret_cast<const float4*>(red + N * k + r);
          alpha[r] = max_nan(max_nan(m[0].x, m[1].x), max_nan(m[2].x, m[3].x));
          alpha[r + 1] = max_nan(max_nan(m[0].y, m[1].y), max_nan(m[2].y, m[3].y));
          alpha[r + 2] = max_nan(max_nan(m[0].z, m[1].z), max_nan(m[2].z, m[3].z));
          alpha[r + 3] = max_nan(max_nan(m[0].w, m[1].w), max_nan(m[2].w, m[3].w));
        }
        // (a row that has seen no key has no reference: its scores are the plain ones, down = 0)
#pragma unroll
        for (int r = 0; r < N; ++r) {
          const bool had = (seen >> r) & 1;
          const float mx = alpha[r];
          const float up = had ? (mx <= kPLog2 ? 0.f : mx - kPLog2) : (mx == kNegInf ? 0.f : mx - kPLog2);
          if (mx != kNegInf) seen |= 1u << r;
          alpha[r] = had ? fast_exp2(-up) : 1.f;
          down[r] -= up;
          y[r] -= up;
          l[r] *= alpha[r];
        }
        if (j > s.pb) {  // O is complete up to the tile before
          ok = mbar_wait(bars.done + 2 * ((i - 1) & 1) + 1, ((i - 1) >> 1) & 1, wd);
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 12; ++c) {
            const uint32_t col = taddr + C::kOCol + R * c + N * half;
            float o[N];
            tmem_ld(col, o);
            tmem_ld_wait();
#pragma unroll
            for (int r = 0; r < N; ++r) o[r] *= alpha[r];
            tmem_st(col, o);
          }
          tmem_st_wait();
        }
      }
      if (C::kPBufs == 1 && i > 0) ok = ok && mbar_wait(bars.done + 2 * ((i - 1) & 1) + 1, ((i - 1) >> 1) & 1, wd);
      const uint32_t pt = smem_u32(smem) + C::kPOff + (i % C::kPBufs) * C::kPBytes + (32 * quarter + lane) * 16 +
                          (N == 8 ? 8 * half : 2048 * half);
#pragma unroll
      for (int r = 0; r < N; ++r) {
        y[r] = fast_exp2(y[r]);
        l[r] += y[r];
      }
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        uint32_t code[N / 2];
#pragma unroll
        for (int r = 0; r < N; r += 2) {
          code[r / 2] = e5m2x2(y[r], y[r + 1]);
          if (term < 2) {
            const uint32_t h2 = e5m2x2_to_f16x2(code[r / 2]);
            y[r] = (y[r] - f16x2_half_to_f32(h2, 0)) * kPStep;
            y[r + 1] = (y[r + 1] - f16x2_half_to_f32(h2, 1)) * kPStep;
          }
        }
        const uint32_t at = pt + term * (R / 16) * 2048;
        if constexpr (N == 8)
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(code[0] | (code[1] << 16)),
                       "r"(code[2] | (code[3] << 16))
                       : "memory");
        else
          st_shared_v4(at, code[0] | (code[1] << 16), code[2] | (code[3] << 16), code[4] | (code[5] << 16),
                       code[6] | (code[7] << 16));
      }
      fence_proxy_async_smem();
      tc_fence_before();
      arrive_warp(bars.p_full + b);
    }

    // row sums, then the rows
    float* red = red2 + (i & 1) * 4 * R;
    float* const lse = reinterpret_cast<float*>(smem + C::kLseOff) + N * half;
    {
      const float sum = reduce_rows<N>(l, lane, add);
      if (lane % (32 / N) == 0) red[N * quarter + lane / (32 / N)] = sum;
      if (quarter == 0 && lane == 0) {
#pragma unroll
        for (int r = 0; r < N; ++r) lse[r] = down[r];
      }
    }
    ok = mbar_wait(bars.done + 2 * ((i - 1) & 1) + 1, ((i - 1) >> 1) & 1, wd);
    tc_fence_after();
    if (!named_bar_and(kHalfBar + half, 128, ok)) return;
    const bool whole = s.pb == 0 && s.pe == s.walk.pages;
    const bool final_out = whole && p.cluster == 0;
    const int slot = piece_slot(whole, prob, 2 * p.num_parts, part, prob == rg.rec.p0);
    const bool slot_ok = final_out || p.cluster > 0 || (slot >= 0 && slot < p.max_slots);
    if (!slot_ok && sw == 0 && lane == 0) atomicOr(p.status, MLA_DEVICE_BAD_SCHEDULE);
    float* const invs = red2 + ((i + 1) & 1) * 4 * R;  // (maxima of the tile before: read)
    if (quarter == 0 && lane < N) {  // a row per lane
      const float sum = (red[lane] + red[N + lane]) + (red[2 * N + lane] + red[3 * N + lane]);
      invs[lane] = sum == 0.f ? 0.f : 1.f / sum;
      const float z = sum == 0.f ? kNegInf : log2f(sum) - lse[lane];
      const int row = g * R + N * half + lane;
      if (p.cluster > 0)
        lse[lane] = z;
      else if (row < p.rows && slot_ok)
        (final_out ? p.lse : p.lse_accum)[static_cast<int64_t>(final_out ? prob : slot) * p.rows + row] = z;
    }
    named_bar_sync(kHalfBar + half, 128);
    float inv[N];
#pragma unroll
    for (int r = 0; r < N; r += 4) {
      const float4 v = *reinterpret_cast<const float4*>(invs + r);
      inv[r] = v.x;
      inv[r + 1] = v.y;
      inv[r + 2] = v.z;
      inv[r + 3] = v.w;
    }
    const int rows = slot_ok ? p.rows - (g * R + N * half) : 0;  // rows from this thread's first on
    const int64_t at = (static_cast<int64_t>(final_out ? prob : slot) * p.rows + g * R + N * half) * kDv + 32 * quarter + lane;
    float* const shared = reinterpret_cast<float*>(smem) + N * half * kDv + 32 * quarter + lane;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float o[N];
      {
        float a[N], z[N];
        const uint32_t col = taddr + C::kOCol + 3 * R * c + N * half;
        tmem_ld(col, o);
        tmem_ld(col + R, a);
        tmem_ld(col + 2 * R, z);
        tmem_ld_wait();
#pragma unroll
        for (int r = 0; r < N; ++r) o[r] = fmaf(fmaf(z[r], 1.f / kPStep, a[r]), 1.f / kPStep, o[r]) * inv[r];
      }
      if (c == 3) {
        tc_fence_before();
        arrive_warp(bars.o_free);
      }
      if (p.cluster > 0) {
#pragma unroll
        for (int r = 0; r < N; ++r) shared[r * kDv + 128 * c] = o[r];
      } else if (final_out) {
        __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + at + 128 * c;
#pragma unroll
        for (int r = 0; r < N; ++r)
          if (r < rows) to[r * kDv] = __float2bfloat16_rn(o[r]);
      } else {
        float* to = p.o_accum + at + 128 * c;
#pragma unroll
        for (int r = 0; r < N; ++r)
          if (r < rows) to[r * kDv] = o[r];
      }
    }
    if (!named_bar_and(kHalfBar + half, 128, true)) return;  // the sums have been read
  }
}

template <int R>
__global__ void __launch_bounds__(kThreads, 1)
    fp4_decode_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_rope,
                      const __nv_bfloat16* __restrict__ q, const DecodeParams p) {
  using C = Cfg<R>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::kMiscOff + 4);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  const Bars bars{bar,
                  bar + C::kRaw,
                  bar + 2 * C::kRaw,
                  bar + 2 * C::kRaw + 2,
                  bar + 2 * C::kRaw + 6,
                  bar + 2 * C::kRaw + 8,
                  bar + 2 * C::kRaw + 10,
                  bar + 2 * C::kRaw + 14};
  // (clusters: `part` is the problem)
  const int unit = p.cluster > 0 ? blockIdx.x / p.cluster : blockIdx.x;
  const int part = unit / p.row_groups, g = unit % p.row_groups;
  if (C::kSmemBytes == C::kBarOff + C::kNumBars * 8 && smem != smem_raw) {
    if (tid == 0) atomicOr(p.status, MLA_DEVICE_BAD_SCHEDULE);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < C::kRaw; ++i) {
      mbar_init(bars.raw_full + i, 1);
      mbar_init(bars.raw_empty + i, kConvWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars.rope_full + i, 1);
      mbar_init(bars.s_full + i, 1);
      mbar_init(bars.p_full + i, kSoftWarps);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bars.k_full + i, kConvWarps);
      mbar_init(bars.done + i, 1);
    }
    mbar_init(bars.o_free, kSoftWarps);
    *abort_flag = 0;
    *reinterpret_cast<volatile int*>(smem + C::kMiscOff + 8) = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_codes);
    tma_prefetch_desc(&tm_rope);
  }
  // (clusters: of a CTA without pages, or one that a wait ran out in)
  if (tid >= 32 && tid < 32 + R) reinterpret_cast<float*>(smem + C::kLseOff)[tid - 32] = kNegInf;
  if (warp == 2) {
    tmem_alloc(const_cast<uint32_t*>(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Watchdog wd{abort_flag, p.status, p.timeout_ns};
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const PartRecord rec = p.cluster > 0 ? cluster_share(p, part) : inline_schedule<false>(p, part, kTile, smem, g == 0);
  const Range rg{rec, rec.p1 < p.num_problems ? rec.p1 : p.num_problems - 1};
  if (warp < 4) {
    regs_to<C::kRegsCtl, kLaunchRegs>();
    if (warp == 0) copy_codes<R>(&tm_codes, p, rg, smem, bars, wd);
    if (warp == 1) score_products<R>(p, rg, tmem, smem, bars, wd);
    if (warp == 2) copy_rope<R>(&tm_rope, p, rg, smem, bars, wd);
    if (warp == 3) value_products<R>(p, rg, tmem, smem, bars, wd);
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, C::kTmemCols);
    if (p.cluster > 0) cluster_merge_wait();
  } else {
    if (warp < 4 + kConvWarps) {
      regs_to<C::kRegsConv, kLaunchRegs>();
      convert<R>(q, p, rg, g, smem, bars, wd);
    } else {
      regs_to<C::kRegsSoft, kLaunchRegs>();
      softmax<R>(p, rg, g, part, tmem, smem, bars, wd);
      tc_fence_before();
    }
    __syncthreads();
    if (p.cluster > 0) {
      const int64_t row = static_cast<int64_t>(part) * p.rows + g * R;
      cluster_merge(p.cluster,
                    ClusterSide{smem, reinterpret_cast<const int*>(smem + C::kMiscOff + 8),
                                reinterpret_cast<const float*>(smem + C::kLseOff)},
                    reinterpret_cast<float*>(smem + C::kPOff), min(R, p.rows - g * R),
                    static_cast<__nv_bfloat16*>(p.out) + row * kDv, p.lse + row);
    }
  }
}

template <int R>
cudaError_t launch(const CUtensorMap& tm_codes, const CUtensorMap& tm_rope, const void* q, const DecodeParams& p,
                   cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.cluster > 0 ? p.cluster * p.num_problems : p.num_parts) * p.row_groups);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<R>::kSmemBytes;
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
  return cudaLaunchKernelEx(&cfg, fp4_decode_kernel<R>, tm_codes, tm_rope, static_cast<const __nv_bfloat16*>(q), p);
}

template <int R>
cudaError_t ready(KernelRegs* regs) {
  auto kern = fp4_decode_kernel<R>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<R>::kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kern);
  if (e == cudaSuccess) *regs = KernelRegs{R == 16 ? "fp4_decode_kernel<16>" : "fp4_decode_kernel<32>", fa.numRegs, kLaunchRegs};
  return e;
}

}  // namespace

cudaError_t launch_decode_fp4(const CUtensorMap& tm_codes, const CUtensorMap& tm_rope, const void* q, const DecodeParams& p,
                              int rpc, cudaStream_t stream) {
  return rpc == 16 ? launch<16>(tm_codes, tm_rope, q, p, stream) : launch<32>(tm_codes, tm_rope, q, p, stream);
}

cudaError_t ready_decode_fp4(int rpc, KernelRegs* regs) { return rpc == 16 ? ready<16>(regs) : ready<32>(regs); }

}  // namespace mla
