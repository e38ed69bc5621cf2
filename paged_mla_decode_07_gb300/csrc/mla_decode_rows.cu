// K9 — windowed decode, 16 query rows per CTA, on register-level matrix
// instructions, over the bf16 cache and both FP8 caches.
//
// Operands go from shared memory straight into the registers of mma.sync:
//     S[r, t] = Q[r, :] . K[t, :]
//     O[r, d] = sum_t P[r, t] V[t, d]
// At 16 rows the legacy matrix instructions (8 cycles for 16 x 8 x 16 per SM
// quarter, measured) need 544 instructions per page, 1.1k cycles, a third of
// what a bf16 page's bytes take; and no TMEM, descriptors, proxy fences or
// issuing warps stand between a copy and its results, which is what the
// smallest calls wait for.  More rows run as groups of 16 that each read the
// pages (from L2).
//
// FP8 rows are never written back to shared memory as bf16 (the tcgen05 kernel's
// load -> dequantise -> multiply chain over one set of slots takes ~5.1k cycles
// per page, where a page's bytes at the card's copy rate take ~1.9k):
//     K[t, d] = bf16_rn(c[t, d] s_b[t])                 (d in block b)
//     O[r, d] = sum_t (P[r, t] s_b[t]) c[t, d]
// Keys are dequantised in registers, as the format defines them.  Values are
// not: their scale joins the probability before it is rounded to bf16 and the
// codes are exact in bf16.  The product keeps one of the two roundings that a
// dequantised value and a rounded P would have.  bf16 and not fp16, although
// fp16 would round less: tokens' scales may lie many orders apart (an all-zero
// tile is stored with scale 1, its neighbours with 1e-6), and P s of the small
// ones has to keep its bits.
//
// Roles (640 threads, registers split by setmaxnreg):
//   warp 0       producer: an FP8 page is one bulk copy of its 64 whole rows
//                (per-token scales come by cp.async), half a bf16 page nine
//                TMA boxes
//   warps 4-11   scores and softmax: warp w owns 16 tokens of the page and half
//                of the dims (FP8: two of the four 128-dim blocks and half of
//                the RoPE dims), with its half of Q as operand fragments in
//                registers; the two halves of a sum meet through shared memory,
//                each warp taking eight of the sixteen rows on
//   warps 12-19  values: warp w owns 64 value dims of all tokens, its 16 x 64
//                part of O in registers
// Score and value warps work on different pages at the same time; P (fp32)
// passes between them through a double buffer.
//
// Measured, 128 elements x 1.1k to 4.2k keys (3.8k on average): bf16 110 us (5.1
// TB/s, 76 % of the copy rate; the tcgen05 kernel 112), FP8 138 us (2.4 TB/s, 35
// %; 175), ~4.4k cycles per page.  FP8 is bound by instruction issue: ~3k warp
// instructions per page and SM quarter, of which two codes cost 6-8 on the score
// side (9 cycles of the conversion and arithmetic pipes, measured alone) and 3 on
// the value side.  Tried: four score warps over whole rows, 5.7k cycles per page
// (latency); sixteen over one block each, 4.5k (issue slots 65 % busy, DRAM 33 %).
// 4 elements x 512 keys: bf16 12.4 us, FP8 13.4.
#include "mla_cluster.cuh"
#include "mla_device.cuh"
#include "mla_internal.h"
#include "mla_schedule.cuh"

namespace mla {
namespace {

constexpr int kRows = 16;
constexpr int kStages = 5;
// Row formats: 656 bytes with four scales, 640 bytes and a scale per token
// elsewhere, 576 bf16.
constexpr int kTile = 0, kToken = 1, kBf16 = 2;
// A stage holds a unit of a page.  FP8: all its rows as they lie in the cache
// (with the 64 scales behind them); 656 bytes are 4 words past a multiple of
// the banks' width, so the operand reads below (eight rows at one 16-byte
// column, four rows at eight 4-byte ones) touch every bank once; rows of 640
// bytes cost two and four passes instead.  bf16: half of its rows, so that two
// and a half pages are in flight, as nine chunks of [32 rows][64 dims] with the
// 128-byte swizzle.  (Rows copied one by one to places 1168 bytes apart: 152 us
// where these take 110, 128 elements x 4160 keys.)
template <int FMT>
struct Rows {
  static constexpr int kUnits = FMT == kBf16 ? 2 : 1;  // units of a page
  static constexpr int kTokens = kPageSize / kUnits;
  static constexpr int kRow = FMT == kBf16 ? 2 * kDqk : FMT == kToken ? 640 : kFp8RowBytes;
  static constexpr int kBytes = kTokens * kRow;
  static constexpr int kReaders = 8 / kUnits;  // score warps that read a unit
};
// bf16: dims 8 d .. 8 d + 7 of row t of a stage
__device__ __forceinline__ uint32_t dims_at(int t, int d) {
  return (d >> 3) * (Rows<kBf16>::kTokens * 128) + t * 128 + (((d ^ t) & 7) << 4);
}
constexpr int kScaleOff = Rows<kToken>::kBytes;  // per-token scales
constexpr int kStageBytes = Rows<kTile>::kBytes;
static_assert(kScaleOff + 4 * kPageSize <= kStageBytes && kStageBytes % 128 == 0 &&
                  Rows<kBf16>::kBytes <= kStageBytes && kStageBytes % 1024 == 0,
              "stage layout");
constexpr int kPStride = 72;                 // floats per row of P: 8 rows x 4 lane groups on distinct banks
constexpr int kPOff = kStages * kStageBytes;
constexpr int kPBytes = kRows * kPStride * 4;
constexpr int kAuxOff = kPOff + 2 * kPBytes;
// aux: score sums on their way to the other half [2][8 warps][32 lanes][4], row maxima of the four
// token groups [2][16][4], alpha [2][16], row sums [16][4], 1/sum [16], page state per stage, abort
// flag, barriers
constexpr int kSwapOff = kAuxOff;
constexpr int kMaxOff = kSwapOff + 2 * 8 * 32 * 16;
constexpr int kAlphaOff = kMaxOff + 2 * kRows * 4 * 4;
constexpr int kSumOff = kAlphaOff + 2 * kRows * 4;
constexpr int kInvOff = kSumOff + kRows * 4 * 4;
constexpr int kFlagOff = kInvOff + kRows * 4;
constexpr int kAbortOff = kFlagOff + 8 * 4;
constexpr int kLseOff = kAbortOff + 4;         // [16], clusters
constexpr int kWhereOff = kLseOff + kRows * 4;  // (clusters) offset of the rows of O
constexpr int kBarOff = (kWhereOff + 4 + 15) / 16 * 16;
static_assert(kRows * kDv * 4 <= kStageBytes && kMaxCluster * (kRows + 1) * 4 <= kMaxOff - kSwapOff, "cluster merge");
constexpr int kNumBars = 2 * kStages + 6;
constexpr int kSmemBytes = kBarOff + kNumBars * 8 + 1024;  // + alignment slack
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(schedule_scratch(kMaxProblems) <= kPOff, "a schedule is made where the pages will be");
constexpr int kThreads = 640;
constexpr uint32_t kRegsCtl = 24, kRegsScore = 128, kRegsValue = 96, kLaunchRegs = 96;
// setmaxnreg hands out what the block was launched with and waits for ever for more
static_assert(kRegsCtl + 2 * kRegsScore + 2 * kRegsValue <= 5 * kLaunchRegs && kThreads * kLaunchRegs <= 65536,
              "register split");
// named barriers: the two warps of a token group (four barriers), the four
// warps of a half (two)
constexpr uint32_t kSwapBar = 1, kRowsBar = 5;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kRescale = 8.0f;             // log2 units: P <= 2^8 before the running max is raised
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Code i of two tokens' words -> two bf16, each 2^-120 times its value: the
// code's sign, exponent and mantissa moved to bf16's places (its subnormals
// become bf16's).  prmt puts each code in a half's lower byte and its sign
// (selector + 8) in all of the upper one, so one shift moves both.  (NaN codes
// become 480: the scores are NaN for them already.)
__device__ __forceinline__ uint32_t code_pair(uint32_t w0, uint32_t w1, int i) {
  uint32_t v;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(v) : "r"(w0), "r"(w1), "r"(i * 0x1111 + 0xc480));
  return (v << 4) & 0x87f087f0u;
}
// P s <= 2^8 s is held at 2^80 times its value, so O at 2^-40: scales up to
// 2^39 stay finite and O has all its bits down to 2^-86.
// Elements of few pages add the product of what the rounding of P s left.  The
// error against 64 bits, relative (0.0017 of it the result's own rounding), is
// then 0.0022 at one page, 0.0020 at 16, 0.0019 at 36, and without it 0.0026 at
// one, 0.0022 at 37, 0.0020 at 66, 0.0018 at 200 (bf16 cache: 0.0021, 0.0020,
// 0.0019; 0.0019, 0.0018, 0.0018): past 36 pages no element is further off than
// short ones are.  Elements of all lengths would take 148 us where they take
// 132 (128 of 66 pages); the condition alone costs 4 of those 132, two copies of
// the loop 12.
constexpr int kFewPages = 36;
__device__ __forceinline__ float bf16x2_half(uint32_t v, int h) { return __uint_as_float(h ? v & 0xffff0000u : v << 16); }
constexpr float kPScale = 1208925819614629174706176.0f;  // 2^80
constexpr float kOScale = 1099511627776.0f;              // 2^40
// Shared-memory reads and writes as plain accesses, which the compiler may
// reorder between the (volatile) waits and arrivals: the operand reads of the
// next products then overlap the conversions and products of the last.
template <class T>
__device__ __forceinline__ T lds(const uint8_t* p) {
  return *reinterpret_cast<const T*>(p);
}
template <class T>
__device__ __forceinline__ void sts(uint8_t* p, T v) {
  *reinterpret_cast<T*>(p) = v;
}
// Four 8 x 8 blocks of 16-bit values, transposed: lane l names the 16 bytes of
// row l % 8 of block l / 8 and gets column l / 4 of each, rows 2 (l % 4) and the next.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&v)[4], uint32_t addr) {
  asm("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(addr)
      : "memory");
}
// What a CTA walks: problems p0..p1 of its part and, in each, a run of pages.
struct Walk {
  int p0, t0, p1, t1, np;
  __device__ int last() const { return p1 < np ? p1 : np - 1; }
};
// The pages of an element: those of a shared prefix, if the call has one, then
// those that its window (or, behind a prefix, every own key) needs.
struct Keys {
  int prefix, prefix_len, len;  // prefix pages, prefix keys, own keys
  KeyWalk own;
  int pages;
  __device__ Keys(const DecodeParams& p, int prob) {
    len = p.cache_seqlens[prob];
    own = key_walk(len, p.s_q, p.window, p.sinks, p.block_table_stride);
    prefix = prefix_len = 0;
    if (p.prefix_len) {
      prefix_len = p.prefix_len[0];
      prefix = pages_of(prefix_len, p.prefix_pages);
    }
    pages = prefix + own.pages;
  }
  // logical page of page i, in the prefix or among the element's own
  __device__ __forceinline__ int page(int i) const { return i < prefix ? i : own.page(i - prefix); }
  __device__ __forceinline__ int keys(int i) const { return i < prefix ? prefix_len : len; }
};
__device__ __forceinline__ void range(const Walk& w, int prob, const Keys& k, int& tb, int& te) {
  tb = prob == w.p0 ? w.t0 : 0;
  te = prob == w.p1 ? min(w.t1, k.pages) : k.pages;
}
// Whether some query token of the element sees key t, and whether all keys of a page are seen.
__device__ __forceinline__ bool key_seen(const DecodeParams& p, int t, int L) {
  return t < L && key_in_walk(t, L, p.s_q, p.window, p.sinks);
}
__device__ __forceinline__ bool page_seen_whole(const DecodeParams& p, int page, int L) {
  const int first = page * kPageSize, last = first + kPageSize - 1;
  if (last >= L) return false;
  const int past = L - p.s_q - p.window;
  return p.sinks > past || last < p.sinks || first > past;
}

struct Bars {
  uint64_t* full;     // [kStages] page landed (bulk copy's bytes, 32 lanes' scale copies)
  uint64_t* empty;    // [kStages] 8 score + 8 value warps are done with the page
  uint64_t* p_full;   // [2] P and alpha of a page are written (8 score warps)
  uint64_t* p_empty;  // [2] the value warps have read them
  uint64_t* l_full;   // 1 / row sums of a segment are written (one warp of each half)
  uint64_t* l_empty;  // the value warps have read them
};

__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const Watchdog& wd) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, wd));
}
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// 16-byte aligned bulk copy global -> shared, completing on `bar`.
__device__ __forceinline__ void bulk_load(uint8_t* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// ---------------------------------------------------------------------------
// producer (one warp)
// ---------------------------------------------------------------------------
template <int FMT>
__device__ void produce(const CUtensorMap* tm_kv, const DecodeParams& p, const Walk& w, uint8_t* smem, const Bars& bars,
                        const Watchdog& wd) {
  const int lane = threadIdx.x & 31;
  const uint64_t pol = p.evict_first ? l2_policy_evict_first() : l2_policy_evict_normal();
  volatile int* flags = reinterpret_cast<volatile int*>(smem + kFlagOff);
  int ut = 0;  // units
  for (int prob = w.p0; prob <= w.last(); ++prob) {
    const Keys k(p, prob);
    int tb, te;
    range(w, prob, k, tb, te);
    const int32_t* bt = p.block_table + static_cast<int64_t>(prob) * p.block_table_stride;
    int ids = -1;  // page ids of pages j0 .. j0 + 31 of the walk, one per lane
    for (int j = tb; j < te; ++j) {
      if (((j - tb) & 31) == 0) {
        const int i = j + lane, lp = i < te ? k.page(i) : -1;
        ids = -1;
        if (lp >= 0 && lp < (i < k.prefix ? p.prefix_pages : p.block_table_stride))
          ids = __ldg((i < k.prefix ? p.prefix_table : bt) + lp);
      }
      const int pg = __shfl_sync(0xffffffffu, ids, (j - tb) & 31);
      const bool ok = pg >= 0 && pg < p.num_pages;
      using R = Rows<FMT>;
#pragma unroll 1
      for (int unit = 0; unit < R::kUnits; ++unit, ++ut) {
        const int s = ut % kStages;
        if (ut >= kStages && !wait_warp(bars.empty + s, ((ut / kStages) - 1) & 1, wd)) goto drain;
        uint8_t* dst = smem + s * kStageBytes;
        const uint8_t* src = p.kv_fp8 + static_cast<int64_t>(ok ? pg : 0) * (R::kUnits * R::kBytes) + unit * R::kBytes;
        if (lane == 0) {
          if (!ok) atomicOr(p.status, MLA_DEVICE_BAD_PAGE);
          flags[s] = ok ? 1 : 0;
          // (an unusable page's stage keeps what it holds: all its tokens are masked)
          mbar_arrive_expect_tx(bars.full + s, ok ? R::kBytes : 0);
          if (ok && FMT != kBf16) bulk_load(dst, src, R::kBytes, bars.full + s, pol);
        }
        if constexpr (FMT == kBf16) {
          __syncwarp();
          if (ok && lane < kNumChunks)
            tma_load_3d(dst + lane * (R::kTokens * 128), tm_kv, bars.full + s, 0, lane,
                        pg * kPageSize + unit * R::kTokens, pol);
        }
        if (FMT == kToken) {
          if (ok) {
            const float* sc = p.kv_scales + static_cast<int64_t>(pg) * kPageSize;
            cp_async4(smem_u32(dst + kScaleOff) + 4 * lane, sc + lane);
            cp_async4(smem_u32(dst + kScaleOff) + 4 * (lane + 32), sc + lane + 32);
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bars.full + s)) : "memory");
        }
        __syncwarp();
      }
    }
  }
drain:
  // no copy may be in flight when the CTA ends, after a timeout either: wait
  // (bounded) for the latest phase of each stage
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (lane == 0) {
    for (int i = ut > kStages ? ut - kStages : 0; i < ut; ++i) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(bars.full + i % kStages, (i / kStages) & 1))
        if (global_timer_ns() - t0 > wd.limit_ns) break;
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------
// scores and softmax (warps 4-11)
// ---------------------------------------------------------------------------
// Operand order.  In an instruction's 16 products over k, lane group c
// (lane % 4) holds k = 2c, 2c + 1, 2c + 8, 2c + 9.  The order of the dims
// within a sum is free, so lane group c takes dims [32 c, 32 c + 32) of a
// block, four per instruction: 16-byte reads of consecutive codes.
template <int FMT>
__device__ void scores(const __nv_bfloat16* __restrict__ q, const DecodeParams& p, const Walk& w, int g, int part,
                       uint8_t* smem, const Bars& bars, const Watchdog& wd) {
  const int lane = threadIdx.x & 31, sw = (threadIdx.x >> 5) - 4;
  const int tg = sw & 3, half = sw >> 2;  // token group, half of the dims (then rows 8 half .. 8 half + 7)
  const int r = lane >> 2, c = lane & 3;
  volatile int* flags = reinterpret_cast<volatile int*>(smem + kFlagOff);
  if (p.debug_stall) {
    // watchdog test: nothing completes this barrier before this role has run
    const bool ok = named_bar_and(kSwapBar + tg, 64, mbar_wait(bars.l_empty, 0, wd));
    if (!named_bar_and(kRowsBar + half, 128, ok)) return;
  }
  const int row = g * kRows + r + 8 * half;  // the row this lane carries through the softmax
  int jt = 0, seg = 0;
  for (int prob = w.p0; prob <= w.last(); ++prob) {
    const Keys walk(p, prob);
    const int L = walk.len;
    int tb, te;
    range(w, prob, walk, tb, te);
    if (tb >= te) continue;

    // Q fragments of this half's dims: rows r and r + 8 of the group (zeros for rows that do not exist)
    uint32_t qf[18][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int qr = g * kRows + r + 8 * h;
      const bool real = qr < p.rows;
      const uint4* src =
          reinterpret_cast<const uint4*>(q + (static_cast<int64_t>(prob) * p.rows + (real ? qr : 0)) * kDqk);
#pragma unroll
      for (int k = 0; k < 9; ++k) {
        // two instructions' worth.  FP8: block 2 half + k / 4, dims 32 c + 8 (k % 4) of it; the last RoPE dims 16 c +
        // 8 half.  bf16: of this half's 288 dims 64 (k / 2) + 16 c + 8 (k % 2); the last 256 + 8 c
        const int at = FMT == kBf16 ? 36 * half + (k < 8 ? 8 * (k >> 1) + 2 * c + (k & 1) : 32 + c)
                       : k < 8      ? 16 * (2 * half + (k >> 2)) + 4 * c + (k & 3)
                                    : 64 + 2 * c + half;
        const uint4 v = real ? __ldg(src + at) : make_uint4(0, 0, 0, 0);
        qf[2 * k][h] = v.x;
        qf[2 * k][h + 2] = v.y;
        qf[2 * k + 1][h] = v.z;
        qf[2 * k + 1][h + 2] = v.w;
      }
    }
    const int lim = p.is_causal ? min(L - p.s_q + row / p.h_q, L - 1) : L - 1;
    const int low = lim - p.window;  // keys up to here are outside the window
    float m = kNegInf, l = 0.f;

    for (int j = tb; j < te; ++j, ++jt) {
      using R = Rows<FMT>;
      const int ut = R::kUnits * jt + (16 * tg) / R::kTokens;  // the unit that holds the token group
      const int s = ut % kStages, buf = jt & 1;
      bool ok = wait_warp(bars.full + s, (ut / kStages) & 1, wd);
      const uint8_t* stage = smem + s * kStageBytes;
      // operand column r; the next group 8 rows on
      const uint8_t* keys = stage + (16 * tg % R::kTokens + r) * R::kRow;
      // scales of this lane's two key tokens for the two blocks
      float sc[2][2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if (FMT == kToken) {
          sc[n][0] = sc[n][1] = lds<float>(stage + kScaleOff + 4 * (16 * tg + 8 * n + r));
        } else if (FMT == kTile) {
          const float2 v = lds<float2>(keys + 8 * n * kFp8RowBytes + kFp8ScaleOffset + 8 * half);
          sc[n][0] = v.x;
          sc[n][1] = v.y;
        }
      }
      // [token group][row r: tokens 2c, 2c + 1; row r + 8: the same], in two
      // parts so that four chains of products run at a time
      float x[2][4], y[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] = y[n][e] = 0.f;
      if constexpr (FMT == kBf16) {
#pragma unroll
        for (int k = 0; k < 9; ++k)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int d = 36 * half + (k < 8 ? 8 * (k >> 1) + 2 * c + (k & 1) : 32 + c);
            const uint4 v = lds<uint4>(stage + dims_at(16 * (tg & 1) + 8 * n + r, d));
            mma_bf16(x[n], qf[2 * k], v.x, v.y);
            mma_bf16(y[n], qf[2 * k + 1], v.z, v.w);
          }
      } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // block 2 half + k / 2, 16 codes k % 2 of this lane's 32
        uint4 v[2];
#pragma unroll
        for (int n = 0; n < 2; ++n)
          v[n] = lds<uint4>(keys + 8 * n * R::kRow + 128 * (2 * half + (k >> 1)) + 32 * c + 16 * (k & 1));
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t word = i == 0 ? v[n].x : i == 1 ? v[n].y : i == 2 ? v[n].z : v[n].w;
            mma_bf16((i & 1) ? y[n] : x[n], qf[4 * k + i], e4m3x2_scaled_bf16x2(word & 0xffffu, sc[n][k >> 1]),
                     e4m3x2_scaled_bf16x2(word >> 16, sc[n][k >> 1]));
          }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint4 v =
            lds<uint4>(keys + 8 * n * R::kRow + (FMT == kToken ? kDv : kFp8RopeOffset) + 32 * c + 16 * half);
        mma_bf16(x[n], qf[16], v.x, v.y);
        mma_bf16(y[n], qf[17], v.z, v.w);
      }
      }
      const bool page_ok = flags[s] != 0;
      // the other half's rows go to its warp of this token group, this half's come from there.  (A
      // buffer is written again two pages on, after the barriers of the page between.)
      float4* swap = reinterpret_cast<float4*>(smem + kSwapOff) + buf * 8 * 32;
      swap[sw * 32 + lane] = half == 0 ? make_float4(x[0][2] + y[0][2], x[0][3] + y[0][3], x[1][2] + y[1][2], x[1][3] + y[1][3])
                                       : make_float4(x[0][0] + y[0][0], x[0][1] + y[0][1], x[1][0] + y[1][0], x[1][1] + y[1][1]);
      float z[4];  // tokens 2c, 2c + 1, 8 + 2c, 9 + 2c of the group for row r + 8 half
#pragma unroll
      for (int i = 0; i < 4; ++i)
        z[i] = half == 0 ? x[i >> 1][i & 1] + y[i >> 1][i & 1] : x[i >> 1][2 + (i & 1)] + y[i >> 1][2 + (i & 1)];
      arrive_warp(bars.empty + s);  // the page is read
      // the P buffer was last read for the page two back
      if (jt >= 2) ok = wait_warp(bars.p_empty + buf, ((jt >> 1) - 1) & 1, wd) && ok;
      // a warp that gave up tells its partner here and both tell their halves
      // below: all eight leave at the same page
      ok = named_bar_and(kSwapBar + tg, 64, ok);
      {
        const float4 o = swap[(sw ^ 4) * 32 + lane];
        z[0] = (z[0] + o.x) * p.scale_log2;
        z[1] = (z[1] + o.y) * p.scale_log2;
        z[2] = (z[2] + o.z) * p.scale_log2;
        z[3] = (z[3] + o.w) * p.scale_log2;
      }
      // mask: page usable, key at or before the row's last one, and among the first keys or in the window
      const int first = walk.page(j) * kPageSize, last = j < walk.prefix ? walk.prefix_len - 1 : lim;
      if (!(page_ok && first + kPageSize - 1 <= last &&
            (first + kPageSize - 1 < p.sinks || first > low))) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = first + 16 * tg + 2 * c + 8 * (i >> 1) + (i & 1);
          if (!(page_ok && t <= last && (t < p.sinks || t > low))) z[i] = kNegInf;
        }
      }
      // row maximum: the lane groups of the warp, then the four token groups
      float mx = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      uint8_t* tops = smem + kMaxOff + (buf * kRows + r + 8 * half) * 16;
      if (c == 0) sts(tops + 4 * tg, mx);
      if (!named_bar_and(kRowsBar + half, 128, ok)) return;
      const float4 top4 = lds<float4>(tops);
      const float top = fmaxf(fmaxf(top4.x, top4.y), fmaxf(top4.z, top4.w));
      float alpha = 1.f;
      if (top > m + kRescale) {  // (the first finite maximum always)
        alpha = m == kNegInf ? 0.f : fast_exp2(m - top);
        m = top;
        l *= alpha;
      }
      if (tg == 0 && c == 0) sts(smem + kAlphaOff + (buf * kRows + r + 8 * half) * 4, alpha);
      float pr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pr[i] = z[i] == kNegInf ? 0.f : fast_exp2(z[i] - m);
        l += pr[i];
      }
      uint8_t* prow = smem + kPOff + buf * kPBytes + ((r + 8 * half) * kPStride + 16 * tg + 2 * c) * 4;
      sts(prow, make_float2(pr[0], pr[1]));
      sts(prow + 32, make_float2(pr[2], pr[3]));
      arrive_warp(bars.p_full + buf);
    }

    // end of the segment: row sums over lane groups and token groups, 1 / sum for the value warps, the log-sum-exp
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (c == 0) sts(smem + kSumOff + ((r + 8 * half) * 4 + tg) * 4, l);
    bool ok = true;
    if (seg > 0) ok = wait_warp(bars.l_empty, (seg - 1) & 1, wd);  // the previous segment's sums are read
    ok = named_bar_and(kSwapBar + tg, 64, ok);
    if (!named_bar_and(kRowsBar + half, 128, ok)) return;
    if (tg == 0) {
      if (c == 0) {
        const bool whole = tb == 0 && te == walk.pages;
        const bool final_out = whole && !p.always_partial;
        const int slot = piece_slot(whole, prob, 2 * p.num_parts, part, prob == w.p0);
        const float4 v = lds<float4>(smem + kSumOff + (r + 8 * half) * 16);
        const float sum = (v.x + v.y) + (v.z + v.w);
        sts(smem + kInvOff + (r + 8 * half) * 4, sum == 0.f ? 0.f : (FMT == kBf16 ? 1.f : kOScale) / sum);
        const float lse = sum == 0.f ? kNegInf : m + log2f(sum);  // (NaN stays NaN)
        if (p.cluster > 0) {
          sts(smem + kLseOff + (r + 8 * half) * 4, lse);
        } else if (row < p.rows) {
          if (final_out)
            p.lse[static_cast<int64_t>(prob) * p.rows + row] = lse;
          else if (slot >= 0 && slot < p.max_slots)
            p.lse_accum[static_cast<int64_t>(slot) * p.rows + row] = lse;
        }
      }
      arrive_warp(bars.l_full);
    }
    // (the sums are written again only after the next segment's barriers)
    ++seg;
  }
}

// ---------------------------------------------------------------------------
// values (warps 12-19)
// ---------------------------------------------------------------------------
// Warp v owns value dims [64 v, 64 v + 64), half of block v / 2.  Lane (r, c)
// reads four codes at dims 32 g + 4 r of tokens 2c, 2c + 1, 2c + 8, 2c + 9 of a
// 16-token step: column r of the instruction for code i is dim 32 g + 4 r + i, so
// a lane ends with dims 32 g + 8 c .. + 7 of rows r and r + 8: 16-byte stores.
template <int FMT>
__device__ void values(const DecodeParams& p, const Walk& w, int g, int part, uint8_t* smem, const Bars& bars,
                       const Watchdog& wd) {
  const int lane = threadIdx.x & 31, v = (threadIdx.x >> 5) - 12;
  const int r = lane >> 2, c = lane & 3;
  const int blk = v >> 1;
  volatile int* flags = reinterpret_cast<volatile int*>(smem + kFlagOff);
  int jt = 0, seg = 0;
  for (int prob = w.p0; prob <= w.last(); ++prob) {
    const Keys walk(p, prob);
    int tb, te;
    range(w, prob, walk, tb, te);
    if (tb >= te) continue;
    const bool few = FMT != kBf16 && walk.pages <= kFewPages;
    float o[2][4][4];  // [32-dim group][code i][row r: dims 8c + i, 8c + 4 + i; row r + 8]
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[a][i][e] = 0.f;
    for (int j = tb; j < te; ++j, ++jt) {
      using R = Rows<FMT>;
      const int ut = R::kUnits * jt, s = ut % kStages, buf = jt & 1;
      const int s1 = (ut + R::kUnits - 1) % kStages;  // the page's last unit
      if (!wait_warp(bars.full + s, (ut / kStages) & 1, wd)) return;
      if (R::kUnits > 1 && !wait_warp(bars.full + s1, ((ut + 1) / kStages) & 1, wd)) return;
      const uint8_t* stage = smem + s * kStageBytes;
      const int lp = walk.page(j);
      const bool page_ok = flags[s] != 0;
      const int L = walk.keys(j);
      const bool whole = page_ok && page_seen_whole(p, lp, L);
      if (!wait_warp(bars.p_full + buf, (jt >> 1) & 1, wd)) return;
      const uint8_t* pa = smem + kPOff + buf * kPBytes;
      const float a0 = lds<float>(smem + kAlphaOff + (buf * kRows + r) * 4);
      const float a1 = lds<float>(smem + kAlphaOff + (buf * kRows + r + 8) * 4);
      if (__any_sync(0xffffffffu, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[a][i][0] *= a0;
            o[a][i][1] *= a0;
            o[a][i][2] *= a1;
            o[a][i][3] *= a1;
          }
      }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const int t = 16 * kk + 2 * c;
        float2 x[4];  // P of rows r, r + 8 at tokens t, t + 1; then t + 8, t + 9
        x[0] = lds<float2>(pa + (r * kPStride + t) * 4);
        x[1] = lds<float2>(pa + ((r + 8) * kPStride + t) * 4);
        x[2] = lds<float2>(pa + (r * kPStride + t + 8) * 4);
        x[3] = lds<float2>(pa + ((r + 8) * kPStride + t + 8) * 4);
        float2 sl = {}, sh = {};
        if (FMT == kToken) {
          sl = lds<float2>(stage + kScaleOff + 4 * t);
          sh = lds<float2>(stage + kScaleOff + 4 * (t + 8));
        } else if (FMT == kTile) {
          const uint8_t* row = stage + t * kFp8RowBytes + kFp8ScaleOffset + 4 * blk;
          sl = make_float2(lds<float>(row), lds<float>(row + kFp8RowBytes));
          sh = make_float2(lds<float>(row + 8 * kFp8RowBytes), lds<float>(row + 9 * kFp8RowBytes));
        }
        // a token that no row sees may hold anything: its scale and codes become 0
        bool k0 = true, k1 = true, k8 = true, k9 = true;
        if (!whole) {
          const int t0 = lp * kPageSize + t;
          k0 = page_ok && key_seen(p, t0, L), k1 = page_ok && key_seen(p, t0 + 1, L);
          k8 = page_ok && key_seen(p, t0 + 8, L), k9 = page_ok && key_seen(p, t0 + 9, L);
          if (!k0) sl.x = 0.f;
          if (!k1) sl.y = 0.f;
          if (!k8) sh.x = 0.f;
          if (!k9) sh.y = 0.f;
        }
        if constexpr (FMT == kBf16) {
          const uint32_t a[4] = {pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                                 pack_bf16x2(x[3].x, x[3].y)};
          // lane l names row l % 16 of the step's tokens (or of the 8 dims further on, from lane 16)
          const uint32_t rows = smem_u32(smem + (kk < 2 ? s : s1) * kStageBytes);
          const uint32_t m0 = (k0 ? 0xffffu : 0u) | (k1 ? 0xffff0000u : 0u);
          const uint32_t m8 = (k8 ? 0xffffu : 0u) | (k9 ? 0xffff0000u : 0u);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b[4];
            ldmatrix_x4_trans(b, rows + dims_at(16 * (kk & 1) + (lane & 15), 8 * v + 2 * i + (lane >> 4)));
            if (!whole) {
              b[0] &= m0;
              b[1] &= m8;
              b[2] &= m0;
              b[3] &= m8;
            }
            mma_bf16(o[i >> 1][2 * (i & 1)], a, b[0], b[1]);
            mma_bf16(o[i >> 1][2 * (i & 1) + 1], a, b[2], b[3]);
          }
        } else {
          sl.x *= kPScale;
          sl.y *= kPScale;
          sh.x *= kPScale;
          sh.y *= kPScale;
          x[0] = make_float2(x[0].x * sl.x, x[0].y * sl.y);
          x[1] = make_float2(x[1].x * sl.x, x[1].y * sl.y);
          x[2] = make_float2(x[2].x * sh.x, x[2].y * sh.y);
          x[3] = make_float2(x[3].x * sh.x, x[3].y * sh.y);
          uint32_t a[4], rest[4];  // P s and what its rounding left
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = pack_bf16x2(x[i].x, x[i].y);
            if (few) rest[i] = pack_bf16x2(x[i].x - bf16x2_half(a[i], 0), x[i].y - bf16x2_half(a[i], 1));
          }
          constexpr int kRow = R::kRow;
          const uint8_t* codes = stage + t * kRow + 64 * v + 4 * r;
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            uint32_t w0 = lds<uint32_t>(codes + 32 * d), w1 = lds<uint32_t>(codes + 32 * d + kRow);
            uint32_t w8 = lds<uint32_t>(codes + 32 * d + 8 * kRow), w9 = lds<uint32_t>(codes + 32 * d + 9 * kRow);
            if (!whole) {
              if (!k0) w0 = 0;
              if (!k1) w1 = 0;
              if (!k8) w8 = 0;
              if (!k9) w9 = 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t b0 = code_pair(w0, w1, i), b1 = code_pair(w8, w9, i);
              mma_bf16(o[d][i], a, b0, b1);
              if (few) mma_bf16(o[d][i], rest, b0, b1);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bars.p_empty + buf);
        mbar_arrive(bars.empty + s);
        if (R::kUnits > 1) mbar_arrive(bars.empty + s1);
      }
    }

    if (!wait_warp(bars.l_full, seg & 1, wd)) return;
    const float i0 = lds<float>(smem + kInvOff + r * 4), i1 = lds<float>(smem + kInvOff + (r + 8) * 4);
    arrive_warp(bars.l_empty);
    const bool piece_whole = tb == 0 && te == walk.pages;
    const bool final_out = piece_whole && !p.always_partial;
    const int slot = piece_slot(piece_whole, prob, 2 * p.num_parts, part, prob == w.p0);
    const bool slot_ok = final_out || p.cluster > 0 || (slot >= 0 && slot < p.max_slots);
    // (clusters: rows for the merge go to the stage that the next page would
    // take; the value warps are at most two pages apart, so none reads it)
    const int free_at = Rows<FMT>::kUnits * jt % kStages * kStageBytes;
    uint8_t* rows_at = smem + free_at;
    if (p.cluster > 0 && v == 0 && lane == 0) sts(smem + kWhereOff, free_at);
    if (!slot_ok && lane == 0) atomicOr(p.status, MLA_DEVICE_BAD_SCHEDULE);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = g * kRows + r + 8 * h;
      if (!slot_ok || row >= p.rows) continue;
      const float inv = h == 0 ? i0 : i1;
      const int64_t at = (static_cast<int64_t>(final_out ? prob : slot) * p.rows + row) * kDv + 64 * v;
      if constexpr (FMT == kBf16) {
        // dims 8 t + 2 c, 8 t + 2 c + 1
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const float y0 = o[t >> 2][t & 3][2 * h] * inv, y1 = o[t >> 2][t & 3][2 * h + 1] * inv;
          const int d = 8 * t + 2 * c;
          if (p.cluster > 0)
            sts(rows_at + ((r + 8 * h) * kDv + 64 * v + d) * 4, make_float2(y0, y1));
          else if (final_out)
            *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + at + d) = pack_bf16x2(y0, y1);
          else
            *reinterpret_cast<float2*>(p.o_accum + at + d) = make_float2(y0, y1);
        }
      } else {
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          float y[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[i] = o[d][i][2 * h] * inv;
            y[4 + i] = o[d][i][2 * h + 1] * inv;
          }
          if (p.cluster > 0) {
            uint8_t* dst = rows_at + ((r + 8 * h) * kDv + 64 * v + 8 * c + 32 * d) * 4;
            sts(dst, make_float4(y[0], y[1], y[2], y[3]));
            sts(dst + 16, make_float4(y[4], y[5], y[6], y[7]));
          } else if (final_out) {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at + 8 * c + 32 * d) = make_uint4(
                pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
          } else {
            uint32_t z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = __float_as_uint(y[i]);
            st_global_v8(p.o_accum + at + 8 * c + 32 * d, z);
          }
        }
      }
    }
    ++seg;
  }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    rows_kernel(const __grid_constant__ CUtensorMap tm_kv, const __nv_bfloat16* __restrict__ q, const DecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + kBarOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kAbortOff);
  Bars bars{bar, bar + kStages, bar + 2 * kStages, bar + 2 * kStages + 2, bar + 2 * kStages + 4, bar + 2 * kStages + 5};
  const int warp = threadIdx.x >> 5;
  // (clusters: `part` is the problem)
  const int unit = p.cluster > 0 ? blockIdx.x / p.cluster : blockIdx.x;
  const int part = unit / p.row_groups, g = unit % p.row_groups;
  // (clusters: of a CTA without pages, or one that a wait ran out in)
  if (threadIdx.x >= 32 && threadIdx.x < 32 + kRows) sts(smem + kLseOff + (threadIdx.x - 32) * 4, kNegInf);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bars.full + i, FMT == kToken ? 1 + 32 : 1);  // the arming arrival and each lane's scale copies
      mbar_init(bars.empty + i, Rows<FMT>::kReaders + 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars.p_full + i, 8);
      mbar_init(bars.p_empty + i, 8);
    }
    mbar_init(bars.l_full, 2);
    mbar_init(bars.l_empty, 8);
    *abort_flag = 0;
    *reinterpret_cast<int*>(smem + kWhereOff) = 0;
    fence_barrier_init();
  }
  __syncthreads();
  Watchdog wd{abort_flag, p.status, p.timeout_ns};
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const PartRecord rec = p.cluster > 0 ? cluster_share(p, part) : inline_schedule(p, part, kPageSize, smem, g == 0);
  const Walk w{rec.p0, rec.t0, rec.p1, rec.t1, p.num_problems};
  if (warp < 4) {
    regs_to<kRegsCtl, kLaunchRegs>();
    if (warp == 0) produce<FMT>(&tm_kv, p, w, smem, bars, wd);
    __syncthreads();
    if (p.cluster > 0) cluster_merge_wait();
  } else {
    if (warp < 12) {
      regs_to<kRegsScore, kLaunchRegs>();
      scores<FMT>(q, p, w, g, part, smem, bars, wd);
    } else {
      regs_to<kRegsValue, kLaunchRegs>();
      values<FMT>(p, w, g, part, smem, bars, wd);
    }
    __syncthreads();
    if (p.cluster > 0) {
      const int64_t row = static_cast<int64_t>(part) * p.rows + g * kRows;
      cluster_merge(p.cluster,
                    ClusterSide{smem, reinterpret_cast<const int*>(smem + kWhereOff),
                                reinterpret_cast<const float*>(smem + kLseOff)},
                    reinterpret_cast<float*>(smem + kSwapOff), min(kRows, p.rows - g * kRows),
                    static_cast<__nv_bfloat16*>(p.out) + row * kDv, p.lse + row);
    }
  }
}

template <int FMT>
cudaError_t launch(const CUtensorMap& tm_kv, const void* q, const DecodeParams& p, cudaStream_t stream) {
  auto kern = rows_kernel<FMT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != static_cast<int>(kLaunchRegs)) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.cluster > 0 ? p.cluster * p.num_problems : p.num_parts) * p.row_groups);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
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
  return cudaLaunchKernelEx(&cfg, kern, tm_kv, static_cast<const __nv_bfloat16*>(q), p);
}

}  // namespace

cudaError_t launch_decode_rows(const CUtensorMap& tm_kv, const void* q, const DecodeParams& p, bool is_fp8,
                               cudaStream_t stream) {
  if (!is_fp8) return launch<kBf16>(tm_kv, q, p, stream);
  return p.kv_scales ? launch<kToken>(tm_kv, q, p, stream) : launch<kTile>(tm_kv, q, p, stream);
}

}  // namespace mla
