// K13 — attention over whole prompts, packed, causal, with grouped heads: the form
// that MLA prefill has before its up-projections are absorbed.  Queries and keys
// are 192 wide (128 values per head and 64 RoPE values, which a key's heads
// share), values 128.
//
//   out[i, h] = sum_t softmax_t(scale q[i, h] . (k_nope[t, h'], k_rope[t])) v[t, h']
//
// over the keys t of i's sequence (h' = h / (heads per KV head)); causal, query i
// of n sees the first m - n + i + 1 of m keys.
//
// An item is 256 query rows of one head of one sequence, two halves of 128 rows
// (M of the MMAs), over tiles of 128 keys.  The halves share the keys and take
// turns on the tensor pipe: while one has its softmax the other's products run.
//   S [128, 128 keys] = Q [128, 192] K^T    12 MMAs
//   O [128, 128]     += P [128, 128 keys] V  8 MMAs, P from tensor memory
// Tensor memory: S and O of both halves, 512 columns; P takes the place of S.
// Shared memory: Q 96 KB and a ring of eight 16 KB chunks (128 keys x 64 dims),
// three for the keys of a tile and two for its values, each freed on its own.
//
// Bound by the tensor pipe: 20 MMAs of 64 cycles for 128 x 128 pairs of a head,
// 10.5 MFLOP in 1280 cycles, and by the chain of a half: products of S (780 cycles
// and ~150 of latency), softmax (1380), products of O (520 and ~250).  16384 tokens
// x 16 heads take 825 to 860 us, 1600 to 1670 TFLOP/s: 85 to 88 % of the library's
// bf16 rate in bursts, 97 % of its sustained one (tensor pipe active 70.5 %).  On the
// way: products from one warp 1242 TFLOP/s, from a warp each for S and O 1281, all of
// a tile's from one election with 32-bit descriptors 1429, the wait for O's products
// last 1573, Q of each half reloaded on its own 1619.
//
// Short prompts are bound by what lies between two items of a CTA, which is code
// that runs once an item, at the rate that its instructions are fetched (the roles
// of 12 warps do not fit the first caches): 32 prompts of 256 rows x 128 heads took
// 207 us, with a loop over the results 194, waits of half the length, masks from bits
// and the sign of the scale in the products 189, the products of O and the loads of Q
// written once for both halves 185 (not those of S: 16384 tokens 830 -> 925).  5
// prompts of 333 to 4096 rows x 128 heads, each with keys of its own, take 1080 us in
// one call alone and 1225 each in a stream of calls; 955 (alone) where 16 heads share
// their keys.  No two of the 152 items that run at a time do otherwise, so a key tile
// comes from memory for every 256 query rows: 6 GB, which a copy would take 890 us for.
// Not kept there: keys and values brought into L2 one to four tiles
// ahead (1120 to 1160), heads in groups whose keys fit L2 (1232), results transposed
// in registers to store whole lines (32 x 256 rows: 202).
//
// P is rounded to bf16 for the products of O: 8 significant bits, fp32's exponents, so
// that no weight is too small to be held.  The row sums have it in fp32.  A second term
// would be 8 more MMAs on the pipe that bounds the kernel (20 -> 28 a tile); relative
// error of the result 0.0019 to 0.0021 against 0.0015 to 0.0016 of fp32 throughout.
//
// Persistent: the plan kernel sorts the blocks of 256 rows of all sequences by
// their number of key tiles, the CTAs take items from that list, longest first,
// by a counter.  Calls with no more items than SMs have no plan: each CTA finds its
// one item itself, or where there are several SMs for an item a run of its key
// tiles, and the merge kernel joins the runs' results.  Every wait is bounded
// (watchdog).
#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kHeadV = 128;
constexpr int kBlock = kPromptBlock;  // query rows of an item
constexpr int kHalfRows = 128, kKeys = 128;
constexpr int kChunkBytes = 128 * 128;  // 128 rows of 64 bf16 values
constexpr int kSlots = 8, kKChunks = 3, kVChunks = 2, kTileChunks = kKChunks + kVChunks;
constexpr int kQOff = 0;
constexpr int kRingOff = 2 * kKChunks * kChunkBytes;
constexpr int kAuxOff = kRingOff + kSlots * kChunkBytes;
constexpr int kItemInts = 10;
constexpr int kItemOff = kAuxOff;  // [2] items
constexpr int kMiscOff = kItemOff + 2 * kItemInts * 4;
constexpr int kBarOff = kMiscOff + 16;
constexpr int kNumBars = 2 * kSlots + 2 + 2 + 2 + 2 + 2 + 2 + 2 + 2 + 2;
constexpr int kSmemBytes = kBarOff + kNumBars * 8 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory");
constexpr int kThreads = 384;
constexpr uint32_t kRegsCtl = 88, kRegsSoft = 208, kLaunchRegs = 168;
// setmaxnreg hands out what the block was launched with and waits for ever for more
static_assert(kRegsCtl + 2 * kRegsSoft <= 3 * kLaunchRegs && kThreads * kLaunchRegs <= 65536, "register split");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 0, kOCol = 256;  // 128 columns a half
constexpr float kRescale = 8.f;             // log2 units that a score may pass the reference by before it is raised
constexpr float kNegInf = -__builtin_huge_valf();

struct Item {
  int q0, rows, k0, m, see, head, end;  // see: keys that row 0 sees (causal); end: no more items
  int j0 = 0, j1 = 1 << 30;             // key tiles of this run of the item
  // keys that row r sees
  __device__ __forceinline__ int sees(int r, bool causal) const { return causal ? min(m, see + r) : m; }
  // key tiles of half h
  __device__ __forceinline__ int tiles(int h, bool causal) const {
    const int n = min(rows - kHalfRows * h, kHalfRows);
    if (n <= 0) return 0;
    const int keys = sees(kHalfRows * h + n - 1, causal);
    return keys > 0 ? (keys + kKeys - 1) / kKeys : 0;
  }
  // end of this run's tiles of half h: it has some if that is past j0
  __device__ __forceinline__ int stop(int h, bool causal) const { return min(tiles(h, causal), j1); }
};

struct Bars {
  uint64_t* full;        // [kSlots] a chunk has landed
  uint64_t* empty;       // [kSlots] the products that read it are done
  uint64_t* q_full;      // [2] Q of a half has landed
  uint64_t* q_empty;     // [2] the products that read Q of a half are done
  uint64_t* s_full;      // [2] scores of a half are in tensor memory
  uint64_t* p_full;      // [2] P of a half is written
  uint64_t* pv_done;     // [2] the products of O of a half's tile are done
  uint64_t* o_free;      // [2] O of a half has been read
  uint64_t* item_full;   // [2]
  uint64_t* item_empty;  // [2]
  uint64_t* drained;     // [2] all products of S, of O, are done
};

__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const Watchdog& wd) {
  return __all_sync(0xffffffffu, mbar_wait_short(bar, parity, wd));
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

// Item `n` of this CTA, as the load warp has put it into shared memory.  Each lane
// reads a word, the shuffles use them: the arrival behind them is behind the reads.
__device__ __forceinline__ bool get_item(int n, uint8_t* smem, const Bars& bars, const Watchdog& wd, Item& it) {
  if (!wait_warp(bars.item_full + (n & 1), (n >> 1) & 1, wd)) return false;
  const int lane = threadIdx.x & 31;
  const volatile int* v = reinterpret_cast<const volatile int*>(smem + kItemOff) + (n & 1) * kItemInts;
  const int word = v[lane < kItemInts ? lane : 0];
  auto at = [&](int i) { return __shfl_sync(0xffffffffu, word, i); };
  it = Item{at(0), at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8)};
  arrive_warp(bars.item_empty + (n & 1));
  return !it.end;
}

// ---------------------------------------------------------------------------
// loads, and the items (one thread)
// ---------------------------------------------------------------------------
// Brings a box into L2.
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

struct Maps {
  const CUtensorMap *q, *k_nope, *k_rope, *v;
};
// Sequence b: its rows within those of q, its keys within those of k.
struct Sequence {
  int q0, n, k0, m;
  __device__ __forceinline__ Sequence(const PromptParams& p, int b) {
    auto clamp = [](int v, int most) { return min(max(v, 0), most); };
    q0 = clamp(p.q_offsets[b], p.num_q);
    n = max(clamp(p.q_offsets[b + 1], p.num_q) - q0, 0);
    k0 = clamp(p.k_offsets[b], p.num_k);
    m = max(clamp(p.k_offsets[b + 1], p.num_k) - k0, 0);
  }
  __device__ __forceinline__ int blocks() const { return (n + kBlock - 1) / kBlock; }
};

// Block `at` of all sequences' (one warp), for calls without a plan.  The last
// CTA counts them all: offsets that decrease may name more than the call has CTAs for.
__device__ __forceinline__ Item find_block(const PromptParams& p, int at) {
  const int lane = threadIdx.x & 31;
  const bool count = blockIdx.x == gridDim.x - 1;
  int before = 0;  // blocks of the sequences up to b0
  Item it{0, 0, 0, 0, 0, 0, 1};
  for (int b0 = 0; b0 < p.batch && (it.end || count); b0 += 32) {
    const int b = b0 + lane, n = b < p.batch ? Sequence(p, b).blocks() : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const uint32_t has = __ballot_sync(0xffffffffu, before + sum > at);
    if (has && it.end) {
      const int k = __ffs(has) - 1;
      const Sequence s(p, b0 + k);
      const int row = (at - before - __shfl_sync(0xffffffffu, sum - n, k)) * kBlock;
      it = Item{s.q0 + row, min(kBlock, s.n - row), s.k0, s.m, s.m - s.n + row + 1, 0, 0};
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  if (count && lane == 0 && before > p.max_blocks) atomicOr(p.status, MLA_DEVICE_BAD_SCHEDULE);
  return it;
}

__device__ void load(const Maps& tm, const PromptParams& p, const Item& own, uint8_t* smem, const Bars& bars, const Watchdog& wd) {
  const uint64_t pol = l2_policy_evict_normal();
  const int group = p.h_q / p.h_kv;
  const int total = p.planned ? p.plan[kPromptBlocks] * p.h_q : 0;  // (below 2^31 by the host's check)
  uint32_t chunk = 0;  // chunks of keys and values so far
  int n = 0;
  // An item is taken late, while the last two tiles of the one before are loaded: one
  // taken earlier waits for its turn here where another CTA is free (8 chunks of 256 to
  // 1023 queries behind up to 8192 keys, 16 heads: 231 us for 214).
  int ticket = total;
  int4 e0, e1;
  auto take = [&]() {
    if (p.planned) ticket = atomicAdd(p.plan + kPromptCounter, 1);
  };
  auto look = [&]() {
    if (ticket >= total) return;
    const int4* e = reinterpret_cast<const int4*>(p.plan + kPromptList) + 2 * (ticket / p.h_q);
    e0 = e[0];
    e1 = e[1];
  };
  auto item = [&]() {
    return ticket >= total ? Item{0, 0, 0, 0, 0, 0, 1} : Item{e0.x, e0.y, e0.z, e0.w, e1.x, ticket % p.h_q, 0};
  };
  take();
  look();
  Item next = p.planned ? item() : own;
#pragma unroll 1
  for (;; ++n) {
    const Item it = next;
    if (n >= 2 && !mbar_wait_short(bars.item_empty + (n & 1), ((n >> 1) - 1) & 1, wd)) break;
    volatile int* v = reinterpret_cast<volatile int*>(smem + kItemOff) + (n & 1) * kItemInts;
    v[0] = it.q0;
    v[1] = it.rows;
    v[2] = it.k0;
    v[3] = it.m;
    v[4] = it.see;
    v[5] = it.head;
    v[6] = it.end;
    v[7] = it.j0;
    v[8] = it.j1;
    mbar_arrive(bars.item_full + (n & 1));
    if (it.end) break;
    const int nt = max(it.stop(0, p.causal), it.stop(1, p.causal)), late = max(it.j0, nt - 2);
    bool ok = true;
    const int kv_head = it.head / group;
#pragma unroll 1
    for (int j = it.j0; j < nt && ok; ++j) {
      if (j == late) take();
#pragma unroll 1
      for (int c = 0; c < kTileChunks; ++c, ++chunk) {
        const int slot = chunk % kSlots;
        if (c == 2 && j == nt - 1) look();
        ok = chunk < kSlots || mbar_wait_short(bars.empty + slot, (chunk / kSlots - 1) & 1, wd);
        if (!ok) break;
        mbar_arrive_expect_tx(bars.full + slot, kChunkBytes);
        uint8_t* dst = smem + kRingOff + slot * kChunkBytes;
        const int row = it.k0 + j * kKeys;
        if (c < 2)
          tma_load_3d(dst, tm.k_nope, bars.full + slot, 64 * c, kv_head, row, pol);
        else if (c == 2)
          tma_load_3d(dst, tm.k_rope, bars.full + slot, 0, 0, row, pol);  // (one head)
        else {
          // values 0 .. 63 go to the lower slot of the two (the ring's end lies between them where
          // the first is its last): the MMAs take the second chunk a positive distance behind
          const bool wraps = (chunk - (c - 3)) % kSlots == kSlots - 1;
          tma_load_3d(dst, tm.v, bars.full + slot, 64 * ((c - 3) ^ (wraps ? 1 : 0)), kv_head, row, pol);
        }
      }
    }
    if (!ok) break;
    if (nt <= it.j0) {
      take();
      look();
    }
    next = item();
    if (!next.end)
#pragma unroll 1
      for (int h = 0; h < 2; ++h)
        if (next.tiles(h, p.causal) > 0)
#pragma unroll 1
          for (int c = 0; c < kKChunks; ++c) tma_prefetch_3d(tm.q, 64 * c, next.head, next.q0 + kHalfRows * h);
  }
  // no copy may be in flight when the CTA ends
  for (uint32_t i = chunk > kSlots ? chunk - kSlots : 0; i < chunk; ++i) drain(bars.full + i % kSlots, (i / kSlots) & 1, wd);
}

// Q of both halves (one warp): each as soon as the half's last products of the
// item before are done, so that one half starts on an item while the other ends
// the last one.
__device__ void load_queries(const CUtensorMap* tm, const PromptParams& p, uint8_t* smem, const Bars& bars, const Watchdog& wd) {
  const uint64_t pol = l2_policy_evict_normal();
  const int lane = threadIdx.x & 31;
  uint32_t loaded = 0, phase = 3;  // bit h: some were loaded; the parity to wait for (first: that before the first phase)
  bool ok = true;
  Item it;
#pragma unroll 1
  for (int n = 0; ok && get_item(n, smem, bars, wd, it); ++n) {
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      if (it.stop(h, p.causal) <= it.j0) continue;
      ok = ok && wait_warp(bars.q_empty + h, (phase >> h) & 1, wd);
      if (!ok) break;
      phase ^= 1u << h;
      loaded |= 1u << h;
      if (lane == 0) {
        mbar_arrive_expect_tx(bars.q_full + h, kKChunks * kChunkBytes);
#pragma unroll 1
        for (int c = 0; c < kKChunks; ++c)
          tma_load_3d(smem + kQOff + (h * kKChunks + c) * kChunkBytes, tm, bars.q_full + h, 64 * c, it.head,
                      it.q0 + kHalfRows * h, pol);
      }
      __syncwarp();
    }
  }
  if (lane == 0)
#pragma unroll 1
    for (int h = 0; h < 2; ++h)  // (the last load's parity: `phase` has passed it)
      if ((loaded >> h) & 1) drain(bars.q_full + h, (phase >> h) & 1, wd);
  __syncwarp();
}

// ---------------------------------------------------------------------------
// products: those of S (one warp), those of O (one warp)
// ---------------------------------------------------------------------------
// The warps that issue share their schedulers with the softmax warps, so the code
// between two MMAs has to be short (with a wait, an election and 64-bit
// descriptors for every four of them an MMA took 100 cycles to issue, where it
// runs for 64): descriptors are their lower words, the upper word being constant,
// and all MMAs of a tile are issued from one elected thread at a time.
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(kDescHi));
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(kDescHi));
}

__device__ void score_products(const PromptParams& p, uint32_t tmem, uint8_t* smem, const Bars& bars, const Watchdog& wd) {
  const uint32_t base = desc_addr(smem), bars_empty = smem_u32(bars.empty);
  const uint32_t q_lo = desc_lo(base + kQOff, 16), ring_lo = desc_lo(base + kRingOff, 16);
  // (a negative scale: the products are those of -Q, bit 13)
  const uint32_t id_s = idesc_bf16_f32(kHalfRows, kKeys, 0, 0) | (p.scale_log2 < 0.f ? 1u << 13 : 0u);
  uint32_t chunk = 0;  // first chunk of the tile
  int items[2] = {0, 0}, tiles[2] = {0, 0};
  bool ok = true;
  Item it;
#pragma unroll 1
  for (int n = 0; ok && get_item(n, smem, bars, wd, it); ++n) {
    const int nt0 = it.stop(0, p.causal), nt1 = it.stop(1, p.causal), nt = max(nt0, nt1);
#pragma unroll 1
    for (int j = it.j0; j < nt && ok; ++j, chunk += kTileChunks) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (j >= (h ? nt1 : nt0)) continue;
        const bool last_user = h == 1 || j >= nt1;
        if (j == it.j0) ok = ok && wait_warp(bars.q_full + h, items[h]++ & 1, wd);
        if (h == 0 || j >= nt0) {
#pragma unroll
          for (int c = 0; c < kKChunks; ++c)
            ok = ok && wait_warp(bars.full + (chunk + c) % kSlots, ((chunk + c) / kSlots) & 1, wd);
        }
        // P, which lies where S will, has been read (the last wait: each takes about a hundred
        // cycles, and this one ends last)
        ok = ok && (tiles[h] == 0 || wait_warp(bars.pv_done + h, (tiles[h] - 1) & 1, wd));
        ++tiles[h];
        tc_fence_after();
        if (elect_one()) {
          const uint32_t s0 = chunk % kSlots, s1 = (chunk + 1) % kSlots, s2 = (chunk + 2) % kSlots;
          if (ok) {
#pragma unroll
            for (int c = 0; c < kKChunks; ++c) {
              const uint32_t b = ring_lo + (c == 0 ? s0 : c == 1 ? s1 : s2) * (kChunkBytes >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_ss(tmem + kSCol + 128 * h, q_lo + (((h * kKChunks + c) * kChunkBytes) >> 4) + 2 * k, b + 2 * k, id_s,
                        c + k > 0);
            }
          }
          umma_commit(bars.s_full + h);
          if (j == (h ? nt1 : nt0) - 1) umma_commit(bars.q_empty + h);
          if (last_user) {
            umma_commit_u32(bars_empty + 8 * s0);
            umma_commit_u32(bars_empty + 8 * s1);
            umma_commit_u32(bars_empty + 8 * s2);
          }
        }
        __syncwarp();
      }
    }
  }
  // products still running end (or the wait does) before the memory they use is freed
  if (elect_one()) umma_commit(bars.drained);
  __syncwarp();
  drain(bars.drained, 0, wd);
}

__device__ void value_products(const PromptParams& p, uint32_t tmem, uint8_t* smem, const Bars& bars, const Watchdog& wd) {
  const uint32_t base = desc_addr(smem);
  constexpr uint32_t kIdO = idesc_bf16_f32(kHalfRows, kHeadV, 0, 1);
  uint32_t chunk = kKChunks;  // first chunk of the tile's values
  uint32_t o_phase = 3, p_phase = 0;  // bit h: the parity to wait for (of the first O: the phase before the first)
  bool ok = true;
  Item it;
#pragma unroll 1
  for (int n = 0; ok && get_item(n, smem, bars, wd, it); ++n) {
    const int nt0 = it.stop(0, p.causal), nt1 = it.stop(1, p.causal), nt = max(nt0, nt1);
    const int keys = it.sees(it.rows - 1, p.causal);
#pragma unroll 1
    for (int j = it.j0; j < nt && ok; ++j, chunk += kTileChunks) {
      const uint32_t s0 = chunk % kSlots, s1 = (chunk + 1) % kSlots;
      const uint32_t first = min(s0, s1), gap = max(s0, s1) - first;
      const uint32_t b = desc_lo(base + kRingOff + first * kChunkBytes, gap * kChunkBytes);
      const int steps = min(8, (keys - j * kKeys + 15) / 16);  // (rows behind the last key are not read)
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (j >= (h ? nt1 : nt0)) continue;
        const bool last_user = h == 1 || j >= nt1;
        if (j == it.j0) {
          ok = ok && wait_warp(bars.o_free + h, (o_phase >> h) & 1, wd);
          o_phase ^= 1u << h;
        }
        if (h == 0 || j >= nt0)
          ok = ok && wait_warp(bars.full + s0, (chunk / kSlots) & 1, wd) && wait_warp(bars.full + s1, ((chunk + 1) / kSlots) & 1, wd);
        ok = ok && wait_warp(bars.p_full + h, (p_phase >> h) & 1, wd);
        p_phase ^= 1u << h;
        tc_fence_after();
        if (elect_one()) {
          if (ok) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k < steps)
                umma_ts(tmem + kOCol + 128 * h, tmem + kSCol + 128 * h + 8 * k, b + ((k * 16 * 128) >> 4), kIdO, j > it.j0 || k > 0);
          }
          umma_commit(bars.pv_done + h);
          if (last_user) {
            umma_commit(bars.empty + s0);
            umma_commit(bars.empty + s1);
          }
        }
        __syncwarp();
      }
    }
  }
  if (elect_one()) umma_commit(bars.drained + 1);
  __syncwarp();
  drain(bars.drained + 1, 0, wd);
}

// ---------------------------------------------------------------------------
// softmax and results: four warps a half, a row per thread
// ---------------------------------------------------------------------------
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ void tmem_st_words16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ void softmax(const PromptParams& p, uint32_t tmem, uint8_t* smem, const Bars& bars, const Watchdog& wd) {
  const int sw = (threadIdx.x >> 5) - 4, half = sw >> 2, quarter = sw & 3, lane = threadIdx.x & 31;
  const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
  const uint32_t s_at = tmem + lanes + kSCol + 128 * half, o_at = tmem + lanes + kOCol + 128 * half;
  const int r = kHalfRows * half + 32 * quarter + lane;  // row of the item
  const float scale = fmaxf(fabsf(p.scale_log2), 1.1754944e-38f);  // (0 would turn a masked score into NaN)
  const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
  uint32_t tile0 = 0;  // tiles of the CTA before the item
  int n_s = 0;
  Item it;
#pragma unroll 1
  for (int n = 0; get_item(n, smem, bars, wd, it); ++n) {
    const int stop = it.stop(half, p.causal), all_tiles = max(it.tiles(0, p.causal), it.tiles(1, p.causal));
    const bool some = stop > it.j0;
    const int sees = it.sees(r, p.causal), keys = it.sees(it.rows - 1, p.causal);
    float ref = kNegInf, l = 0.f;
    if (p.debug_stall) return;  // watchdog test: the scores are never taken
#pragma unroll 1
    for (int j = it.j0; j < stop; ++j, ++n_s) {
      if (!wait_warp(bars.s_full + half, n_s & 1, wd)) return;
      tc_fence_after();
      float x[kKeys];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float v[32];
        tmem_ld_x32(s_at + 32 * c, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[32 * c + i] = v[i];
      }
      tmem_ld_wait();
      const int valid = sees - j * kKeys;  // of this tile's keys the row sees
      if (__any_sync(0xffffffffu, valid < kKeys)) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int v = valid - 32 * c;
          const uint32_t keep = v >= 32 ? ~0u : v <= 0 ? 0u : (1u << v) - 1;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(keep & (1u << i))) x[32 * c + i] = kNegInf;
        }
      }
      float m0 = max3_nan(x[0], x[1], x[2]), m1 = max3_nan(x[3], x[4], x[5]);
      float m2 = max3_nan(x[6], x[7], x[8]), m3 = max3_nan(x[9], x[10], x[11]);
#pragma unroll
      for (int i = 12; i < kKeys - 4; i += 8) {
        m0 = max3_nan(m0, x[i], x[i + 1]);
        m1 = max3_nan(m1, x[i + 2], x[i + 3]);
        m2 = max3_nan(m2, x[i + 4], x[i + 5]);
        m3 = max3_nan(m3, x[i + 6], x[i + 7]);
      }
      m0 = max3_nan(m0, x[124], x[125]);
      m1 = max3_nan(m1, x[126], x[127]);
      const float top = max_nan(max_nan(m0, m1), max_nan(m2, m3)) * scale;
      const bool raise = !(top <= ref + kRescale);
      if (__any_sync(0xffffffffu, raise)) {
        // (the scores' barrier follows the products of O of the tile before)
        float alpha = 1.f;
        if (raise) {
          alpha = ref == kNegInf ? 1.f : fast_exp2(ref - top);
          ref = top;
          l *= alpha;
        }
        if (j > it.j0) {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            float o[16];
            tmem_ld_x16(o_at + 16 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= alpha;
            tmem_st_x16(o_at + 16 * c, o);
          }
        }
      }
      const float down = ref == kNegInf ? 0.f : -ref;
      float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 y = fma2(make_float2(x[32 * c + 2 * i], x[32 * c + 2 * i + 1]), make_float2(scale, scale),
                          make_float2(down, down));
          y.x = fast_exp2(y.x);
          y.y = fast_exp2(y.y);
          if (i & 1)
            sum1 = add2(sum1, y);
          else
            sum0 = add2(sum0, y);
          w[i] = pack_bf16x2(y.x, y.y);
        }
        tmem_st_words16(s_at + 16 * c, w);
      }
      l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
      if ((j + 1) * kKeys > keys && j == all_tiles - 1 && (keys & 15) != 0) {
        // Rows of V behind the last key that the products read (up to a multiple of 16)
        // belong to other sequences, or to no one: zeros, so that no NaN of theirs
        // meets a weight of 0.  Each half writes them.
        const uint32_t i = (tile0 + j - it.j0) * kTileChunks + kKChunks;
        const int first = keys - j * kKeys, row = first + (threadIdx.x & 127) / 8, unit = threadIdx.x & 7;
        bool ok = true;
#pragma unroll 1
        for (int c = 0; c < 2; ++c)
          ok = ok && wait_warp(bars.full + (i + c) % kSlots, ((i + c) / kSlots) & 1, wd);
        if (!ok) return;
        if (row < ((first + 15) & ~15)) {
#pragma unroll 1
          for (int c = 0; c < 2; ++c)
            st_shared_v4(smem_u32(smem) + kRingOff + ((i + c) % kSlots) * kChunkBytes + row * 128 + unit * 16,
                         0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // (the arrivals of all four warps on P's barrier hand the rows over)
      }
      tmem_st_wait();
      tc_fence_before();
      arrive_warp(bars.p_full + half);
    }
    tile0 += max(max(it.stop(0, p.causal), it.stop(1, p.causal)) - it.j0, 0);

    const bool real = r < it.rows;
    const int64_t row = static_cast<int64_t>(it.q0 + r) * p.h_q + it.head;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * kHeadV;
    if (some) {
      if (!wait_warp(bars.pv_done + half, (n_s - 1) & 1, wd)) return;
      tc_fence_after();
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      float o[32];
      if (some) {
        tmem_ld_x32(o_at + 32 * c, o);
        tmem_ld_wait();
        if (c == 3) {
          tc_fence_before();
          arrive_warp(bars.o_free + half);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0.f;
      }
      if (p.splits > 1) {
        if (real && some) {
          float4* to = reinterpret_cast<float4*>(p.o_part + (static_cast<int64_t>(blockIdx.x) * kBlock + r) * kHeadV + 32 * c);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            to[i] = make_float4(o[4 * i] * inv, o[4 * i + 1] * inv, o[4 * i + 2] * inv, o[4 * i + 3] * inv);
        }
      } else if (real) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = l == 0.f ? 0u : pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
        if (wide) {  // whole sectors: each store instruction costs a pass per row
          st_global_v8(out + 32 * c, {w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]});
          st_global_v8(out + 32 * c + 16, {w[8], w[9], w[10], w[11], w[12], w[13], w[14], w[15]});
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            reinterpret_cast<uint4*>(out)[4 * c + i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
      }
    }
    const float z = l == 0.f ? kNegInf : ref + log2f(l);
    if (p.splits > 1) {
      p.lse_part[static_cast<int64_t>(blockIdx.x) * kBlock + r] = z;
    } else if (real) {
      p.lse[row] = z;
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k_nope,
                  const __grid_constant__ CUtensorMap tm_k_rope, const __grid_constant__ CUtensorMap tm_v,
                  const PromptParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kMiscOff);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kMiscOff + 4);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + kBarOff);
  uint64_t* next = bar;
  auto take = [&](int n) {
    uint64_t* b = next;
    next += n;
    return b;
  };
  Bars bars;
  bars.full = take(kSlots);
  bars.empty = take(kSlots);
  bars.q_full = take(2);
  bars.q_empty = take(2);
  bars.s_full = take(2);
  bars.p_full = take(2);
  bars.pv_done = take(2);
  bars.o_free = take(2);
  bars.item_full = take(2);
  bars.item_empty = take(2);
  bars.drained = take(2);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bars.full + i, 1);
      mbar_init(bars.empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars.q_full + i, 1);
      mbar_init(bars.q_empty + i, 1);
      mbar_init(bars.s_full + i, 1);
      mbar_init(bars.p_full + i, 4);
      mbar_init(bars.pv_done + i, 1);
      mbar_init(bars.drained + i, 1);
      mbar_init(bars.o_free + i, 4);
      mbar_init(bars.item_full + i, 1);
      mbar_init(bars.item_empty + i, 11);  // eight softmax warps, two of products, the one that loads Q
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k_nope);
    tma_prefetch_desc(&tm_k_rope);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 2) {
    tmem_alloc(const_cast<uint32_t*>(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Watchdog wd{abort_flag, p.status, p.timeout_ns};
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp < 4) {
    regs_to<kRegsCtl, kLaunchRegs>();
    if (warp == 0) {
      Item own{0, 0, 0, 0, 0, 0, 1};
      if (!p.planned) {
        const int item = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
        own = find_block(p, item / p.h_q);
        own.head = item % p.h_q;
        if (p.splits > 1) {
          const int nt = max(own.tiles(0, p.causal), own.tiles(1, p.causal));
          own.j0 = nt * split / p.splits;
          own.j1 = nt * (split + 1) / p.splits;
          // for the merge (an item without a block: no rows)
          if (split == 0 && (threadIdx.x & 31) == 0)
            reinterpret_cast<int4*>(p.plan)[item] = make_int4(own.q0, own.rows, own.head, 0);
        }
      }
      if ((threadIdx.x & 31) == 0) load(Maps{&tm_q, &tm_k_nope, &tm_k_rope, &tm_v}, p, own, smem, bars, wd);
      __syncwarp();
    }
    if (warp == 2) load_queries(&tm_q, p, smem, bars, wd);
    if (warp == 1) score_products(p, tmem, smem, bars, wd);
    if (warp == 3) value_products(p, tmem, smem, bars, wd);
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, kTmemCols);
  } else {
    regs_to<kRegsSoft, kLaunchRegs>();
    softmax(p, tmem, smem, bars, wd);
    tc_fence_before();
    __syncthreads();
  }
}

// Joins the runs of an item's rows: a warp per row, four dims per lane.
constexpr int kMergeWarps = 8, kMaxSplits = 16;

__global__ void __launch_bounds__(kMergeWarps * 32) prompt_merge_kernel(const PromptParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, r = blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  const int4 item = reinterpret_cast<const int4*>(p.plan)[blockIdx.y];
  if (r >= item.y) return;
  const int64_t part = static_cast<int64_t>(blockIdx.y) * p.splits * kBlock + r;
  float z[kMaxSplits], top = kNegInf;
#pragma unroll
  for (int k = 0; k < kMaxSplits; ++k) {
    z[k] = k < p.splits ? p.lse_part[part + k * kBlock] : kNegInf;
    top = max_nan(top, z[k]);
  }
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float total = kNegInf;
  if (top != kNegInf) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxSplits; ++k) sum += exp2f(z[k] - top);
    total = top + log2f(sum);
#pragma unroll
    for (int k = 0; k < kMaxSplits; ++k) {
      if (z[k] == kNegInf) continue;  // (no values are there)
      const float4 v = reinterpret_cast<const float4*>(p.o_part + (part + k * kBlock) * kHeadV)[lane];
      const float w = exp2f(z[k] - total);
      o.x += w * v.x;
      o.y += w * v.y;
      o.z += w * v.z;
      o.w += w * v.w;
    }
  }
  const int64_t row = static_cast<int64_t>(item.x + r) * p.h_q + item.z;
  reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + row * kHeadV)[lane] =
      make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  if (lane == 0) p.lse[row] = total;
}

// ---------------------------------------------------------------------------
// the plan: blocks of all sequences, those with the most key tiles first
// ---------------------------------------------------------------------------
// A counting sort over 1024 classes of key tiles in one CTA (the order within a
// class is free: an item's result does not depend on when it runs).  Also sets the
// counter that the items are taken by to zero, so that each call starts it anew.
constexpr int kPlanThreads = 1024, kClasses = 1024;

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PromptParams p) {
  extern __shared__ int first[];  // [batch + 1] blocks of the sequences before
  __shared__ int warp_sum[32], classes[kClasses], most;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int per = (p.batch + kPlanThreads - 1) / kPlanThreads, b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
  // Offsets that decrease may name more blocks than the list has room for, and more than
  // 32 bits hold (16384 sequences of 2^26 rows and of none in turn: 2^31): sums of threads
  // and of warps stop one past the room, so that none of the 32 that are added passes 2^29.
  const int past = p.max_blocks + 1;
  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    first[b] = mine;
    mine = min(mine + Sequence(p, b).blocks(), past);
  }
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = min(x, past);
  if (tid == 0) most = 0;
  classes[tid] = 0;
  __syncthreads();
  if (warp == 0) {
    int t = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    warp_sum[lane] = t;
  }
  __syncthreads();
  const int before = x - mine + (warp > 0 ? warp_sum[warp - 1] : 0);
  for (int b = b0; b < b1; ++b) first[b] += before;
  int total = warp_sum[31];
  if (tid == 0) first[p.batch] = total;
  __syncthreads();
  if (total > p.max_blocks) {
    if (tid == 0) atomicOr(p.status, MLA_DEVICE_BAD_SCHEDULE);
    total = 0;
  }
  // block i: its entry and its key tiles
  auto entry = [&](int i, int4& a, int& see) {
    int lo = 0, hi = p.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= i)
        lo = mid;
      else
        hi = mid - 1;
    }
    const Sequence s(p, lo);
    const int at = (i - first[lo]) * kBlock, rows = min(kBlock, s.n - at);
    a = make_int4(s.q0 + at, rows, s.k0, s.m);
    see = s.m - s.n + at + 1;
    const int keys = p.causal ? min(s.m, see + rows - 1) : s.m;
    return keys > 0 ? (keys + kKeys - 1) / kKeys : 0;
  };
  int longest = 0;
  for (int i = tid; i < total; i += kPlanThreads) {
    int4 a;
    int see;
    longest = max(longest, entry(i, a, see));
  }
  atomicMax(&most, longest);
  __syncthreads();
  int shift = 0;
  while ((most >> shift) >= kClasses) ++shift;
  for (int i = tid; i < total; i += kPlanThreads) {
    int4 a;
    int see;
    atomicAdd(&classes[kClasses - 1 - (entry(i, a, see) >> shift)], 1);
  }
  __syncthreads();
  // places of the classes, the longest first
  int c = classes[tid], z = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, z, o);
    if (lane >= o) z += y;
  }
  if (lane == 31) warp_sum[warp] = z;
  __syncthreads();
  if (warp == 0) {
    int t = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    warp_sum[lane] = t;
  }
  __syncthreads();
  classes[tid] = z - c + (warp > 0 ? warp_sum[warp - 1] : 0);
  __syncthreads();
  int4* list = reinterpret_cast<int4*>(p.plan + kPromptList);
  for (int i = tid; i < total; i += kPlanThreads) {
    int4 a;
    int see;
    const int tiles = entry(i, a, see);
    const int at = atomicAdd(&classes[kClasses - 1 - (tiles >> shift)], 1);
    list[2 * at] = a;
    list[2 * at + 1] = make_int4(see, 0, 0, 0);
  }
  if (tid == 0) {
    p.plan[kPromptCounter] = 0;
    p.plan[kPromptBlocks] = total;
  }
}

}  // namespace

cudaError_t launch_prompt(const CUtensorMap& tm_q, const CUtensorMap& tm_k_nope, const CUtensorMap& tm_k_rope,
                          const CUtensorMap& tm_v, const PromptParams& p, int sm_count, cudaStream_t stream) {
  const int64_t items = static_cast<int64_t>(p.max_blocks) * p.h_q;
  const size_t scratch = (static_cast<size_t>(p.batch) + 1) * sizeof(int);
  cudaError_t e = cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.planned) {
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = scratch;
    e = cudaLaunchKernelEx(&cfg, plan_kernel, p);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(p.planned ? sm_count : items * p.splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  e = cudaLaunchKernelEx(&cfg, prompt_kernel, tm_q, tm_k_nope, tm_k_rope, tm_v, p);
  if (e != cudaSuccess || p.splits == 1) return e;
  cfg.gridDim = dim3(kBlock / kMergeWarps, static_cast<unsigned>(items));
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, prompt_merge_kernel, p);
}

cudaError_t ready_prompt(KernelRegs* regs) {
  cudaError_t e = allow_dynamic_smem(plan_kernel, (kMaxProblems + 1) * sizeof(int), 8192);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, prompt_kernel);
  if (e == cudaSuccess) *regs = KernelRegs{"prompt_kernel", fa.numRegs, kLaunchRegs};
  return e;
}

}  // namespace mla
