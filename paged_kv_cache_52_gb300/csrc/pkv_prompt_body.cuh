// Attention of whole prompts: packed sequences of different lengths, grouped
// heads, K and V as contiguous bf16 rows.  (prompt_attention.cu and
// prompt_attention_shared.cu instantiate the kernel: items of one CTA, items
// that several share.)
//
//   out[i] = softmax(q_i K^T scale) V  over keys 0 .. L - n + i  (all L keys
//   when not causal), i < n the sequence's queries, L its keys (n = L for a
//   prompt; the block-scaled prefill has a cached prefix before its queries).
//
// Two matrix products of 2 n L d flops each per head, half of that under the
// causal mask, over O((n + L) d) bytes: bound by the tensor cores.  Layout:
//  * an item is two tiles of 128 rows -- 128 / G tokens times the G query heads
//    of one KV head each -- against the keys in tiles of 128.  S and O of a row
//    tile stand in tensor memory, P (bf16) is written over S and read from
//    there by the second product.
//  * one CTA per SM works through items for the whole launch: the copies run
//    ahead into the next item, and its first products are issued while the
//    last one's rows are written out.
//  * a thread owns a row in the softmax, its 128 scores in registers: no
//    shuffles, one trip to tensor memory.  The running maximum is looked for
//    only where it has to move: a tile keeps it while every row's weights stay
//    below 2^16 against it, seen from the sum of the first 64 keys' weights and
//    the maximum of the others'.  P leaves in two halves, and the second product
//    starts on the first.  A tile's S is complete only after the product before
//    it, and a row's next P comes only after its O was read, so O needs no
//    barriers of its own.
//  * what waits costs: an mbarrier that is complete takes the MMA warp 135 cycles
//    to see.  So it waits for P alone: the warp that looks after V (below) adds
//    the arrival of the tile's operands to that barrier; V of a tile comes with
//    K of the next, an item's Q with its first K.
//  * P in bf16 is off by 2^-8 of each weight at most, as the bf16 output is of
//    itself; S, O, the weights' sum and the maximum are float32.
//  * where the items are fewer than half the SMs, a cluster of CTAs shares each:
//    every CTA takes a run of its key tiles, and their rows meet through
//    distributed shared memory at the end (one chunk of 8 tokens after 20000:
//    64 heads of 128 on 8: 205 us with one CTA each, 59 so).
//  * items are taken longest first over all sequences (worked out of q_start on
//    the device), heads side by side.
// Keys that no row sees: V rows past a sequence's end, which belong to the next
// one or nobody, are zeroed in shared memory; NaN and infinities of V in the
// tiles that the mask cuts are taken out of the product (0 times them is NaN)
// and added at the end to the rows that see them.
#pragma once

#include <algorithm>
#include <atomic>
#include <climits>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tcgen05.cuh"

namespace pkv {

static __device__ unsigned g_prompt_error = 0;

constexpr int kPrRows = 128;    // rows of a Q tile
constexpr int kPrKeys = 128;    // keys of a K / V tile
constexpr int kPrTiles = 2;     // Q tiles of an item, one softmax warpgroup each
constexpr int kPrThreads = 384; // 2 softmax warpgroups; copies, MMA issue, V scrub, items
// The softmax holds a row's 128 scores: its warps take registers from the others
// (of 384 x 168 that the block is launched with).
constexpr int kPrRegsSoftmax = 200, kPrRegsOther = 104;
static_assert(2 * 128 * kPrRegsSoftmax + 128 * kPrRegsOther <= kPrThreads * 168, "registers");
constexpr int kPrLoadWarp = 8, kPrMmaWarp = 9, kPrScrubWarp = 10, kPrItemWarp = 11;
constexpr float kPrMost = 16.f;  // weights up to 2^16 against the running maximum
// Scores (in log2 units) from which on a row's are rounded as its maximum is before the
// weights: their multiply-add does not share that rounding, half a step of 2^3 here and of
// 2^8 at 2^31, by which all weights of a row would overflow or vanish.
constexpr float kPrLarge = 0x1p26f;
constexpr int kPrRegSets = 16;   // times 32 sequences whose items one warp holds in registers
constexpr int kPrSlots = 4;      // items known ahead
constexpr int kPrMaxSplit = 8;   // CTAs of an item: the portable cluster size

template <int D>
struct PromptCfg {
  static constexpr int kHalf = 128 * 128;             // 128 rows x 64 columns
  static constexpr int kTile = (D / 64) * kHalf;      // of Q, K or V
  // an item's Q and first K (its head), and pairs of a tile's V and the next K
  static constexpr int kHeads = D == 128 ? 1 : 2;
  static constexpr int kPairs = D == 128 ? 2 : 4;
  static constexpr int kHeadTile = (kPrTiles + 1) * kTile, kPairTile = 2 * kTile;
  static constexpr int kPairOff = kHeads * kHeadTile;
  static constexpr int kBarOff = kPairOff + kPairs * kPairTile;
  // barriers: a tile's P in two halves, the first with V and the next K; an
  // item's data in its slot
  static constexpr int kHeadFull = 0, kHeadFree = kHeadFull + kHeads,
                       kPairLand = kHeadFree + kHeads, kPairFree = kPairLand + kPairs,
                       kSFull = kPairFree + kPairs, kPFull = kSFull + kPrTiles,
                       kODone = kPFull + 2 * kPrTiles, kItem = kODone + kPrTiles,
                       kItemFree = kItem + kPrSlots, kDrain = kItemFree + kPrSlots,
                       kNumBars = kDrain + 1;
  static constexpr int kItemOff = kBarOff + kNumBars * 8;
  static constexpr int kMiscOff = kItemOff + kPrSlots * 40;  // tensor memory's base, abort flag
  static constexpr int kSmemBytes = kMiscOff + 16 + 1024;
  // a shared item's rows at its end: O from 0 on, maxima and sums
  static constexpr int kJoinMl = kPrTiles * kPrRows * D * 4;
  static_assert(kJoinMl + kPrTiles * kPrRows * 8 <= kBarOff, "the rings hold an item's rows");
  static constexpr uint32_t kTmemCols = 512, kTileCols = 256;  // S / P, then O at 128
  static_assert(kSmemBytes <= 232448, "shared memory");
};

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// What CTA `rank` of the cluster has at this CTA's shared address `addr`.
template <typename T>
__device__ __forceinline__ T cluster_ld(uint32_t addr, int rank) {
  uint32_t there;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(addr), "r"(rank));
  T v;
  if constexpr (sizeof(T) == 16)
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(there)
                 : "memory");
  else
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(there)
                 : "memory");
  return v;
}

// What the roles need of an item.
struct PromptItem {
  int seq;   // -1: no more
  int kvh, qs, n, keys;
  int t0;    // first query token
  int row0;  // first K / V row
  int j0, j1;  // this CTA's key tiles
  int odd;   // NaN or infinities were taken out of V
};

static_assert(sizeof(PromptItem) == 40, "a slot");

// Bounded wait that also gives up as soon as another role has aborted.
__device__ __forceinline__ bool pr_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  for (uint32_t i = 0; i < kWaitPollLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 255u && *abort_flag) return false;
  }
  return false;
}

__device__ __forceinline__ void pr_abort(volatile int* abort_flag) {
  *abort_flag = 1;
  atomicOr(&g_prompt_error, kErrWaitTimeout);
}

// The lane of a converged warp that issues its MMAs (always the same one).
__device__ __forceinline__ bool elect_lane() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// smem_desc_sw128 (with a stride of 1024 bytes) of a shared address over 16:
// only the low word depends on it, so an operand costs one addition.
template <uint32_t kLbo>
__device__ __forceinline__ uint64_t desc_at(uint32_t addr16) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};"
      : "=l"(d)
      : "r"(addr16 | ((kLbo >> 4) << 16)), "r"((1024u >> 4) | (1u << 14) | (2u << 29)));
  return d;
}

// Bits 15 and 31: which halves of a bf16 pair are NaN or infinite (other bits: anything).
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) {
  return (w & 0x7f807f80u) + 0x00800080u;
}

// Two scores' weights: added to `sum`, and packed as bf16.
__device__ __forceinline__ void weights(float s0, float s1, uint64_t scale2, uint64_t shift2,
                                        uint64_t& sum, uint32_t& packed) {
  float x0, x1;
  f2_unpack(f2_fma(f2_pack(s0, s1), scale2, shift2), x0, x1);
  const float e0 = ex2(x0), e1 = ex2(x1);
  sum = f2_add(sum, f2_pack(e0, e1));
  packed = pack_bf16x2(e0, e1);
}
__device__ __forceinline__ float f2_sum(const uint64_t (&v)[2]) {
  float a, b;
  f2_unpack(f2_add(v[0], v[1]), a, b);
  return a + b;
}

// A sequence's rows and keys; none where they are out of order.
struct PromptSeq {
  int qs, n, keys;
  bool bad;
};
__device__ __forceinline__ PromptSeq prompt_seq(const PromptArgs& p, int s) {
  PromptSeq q;
  q.qs = __ldg(p.q_start + s);
  const int qe = __ldg(p.q_start + s + 1);
  q.n = qe - q.qs;
  q.keys = p.kv_lens ? __ldg(p.kv_lens + s) : q.n;
  q.bad = q.qs < 0 || q.n < 0 || qe > p.total_q ||
          (q.n > 0 && ((p.causal && q.keys < q.n) || q.keys <= 0 ||
                       (p.kv_lens && q.keys > p.kv_stride)));
  if (q.bad) q.n = 0;
  return q;
}

// The items of one sequence: `items` of tpc tokens, causal ones at levels lo,
// lo + 1, ... (the last key over tpc), else all at level lo.
struct PromptLevels {
  int lo, items;
};
__device__ __forceinline__ PromptLevels prompt_levels(const PromptArgs& p, int s, int tpc) {
  const PromptSeq q = prompt_seq(p, s);
  PromptLevels v;
  v.items = (q.n + tpc - 1) / tpc;
  v.lo = v.items == 0 ? 0 : (p.causal ? q.keys - q.n : q.keys) / tpc;
  return v;
}

// Item `rank` of a KV head, by one warp, those with the most keys first: finds
// the level by bisection over the counts of items at or above one, then the
// sequence within it.  `own`: lane l's sequences l, l + 32, ... of the first
// 32 kSets; the others' are worked out again each time.  `seqs`: how many count.
// kSets 1 serves up to 32 sequences with little code, which a first item waits
// for while it is fetched.
template <int kSets>
struct PromptTable {
  PromptLevels own[kSets];
  int seqs;

  __device__ __forceinline__ void load(const PromptArgs& p, int tpc) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
      const int s = i * 32 + lane;
      own[i] = s < seqs ? prompt_levels(p, s, tpc) : PromptLevels{0, 0};
    }
  }
  // f(levels, sequence of lane 0) for every lane's sequences until it is false
  template <typename F>
  __device__ __forceinline__ void each(const PromptArgs& p, int tpc, F&& f) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
      if (kSets > 1 && i * 32 >= seqs) return;
      if (!f(own[i], i * 32)) return;
    }
    if constexpr (kSets > 1)
      for (int s0 = kSets * 32; s0 < seqs; s0 += 32) {
        const int s = s0 + lane;
        if (!f(s < seqs ? prompt_levels(p, s, tpc) : PromptLevels{0, 0}, s0)) return;
      }
  }
  __device__ __forceinline__ bool item(const PromptArgs& p, int tpc, int rank, int& seq,
                                       int& tile) const {
    constexpr unsigned kFull = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    const bool causal = p.causal != 0;
    auto above = [&](const PromptLevels& v, int level) {
      if (!causal) return v.lo >= level ? v.items : 0;
      return min(v.items, max(0, v.lo + v.items - level));
    };
    auto count = [&](int level) {
      int c = 0;  // (the launch's items are within 32 bits)
      each(p, tpc, [&](const PromptLevels& v, int) {
        c += above(v, level);
        return true;
      });
      return __reduce_add_sync(kFull, c);
    };
    int top = 0, all = 0;  // no item at level top
    each(p, tpc, [&](const PromptLevels& v, int) {
      if (v.items > 0) top = max(top, v.lo + (causal ? v.items : 1));
      all += v.items;
      return true;
    });
    top = __reduce_max_sync(kFull, top);
    if (__reduce_add_sync(kFull, all) <= rank) return false;
    int lo = 0, hi = top;  // count(lo) > rank >= count(hi)
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (count(mid) > rank) lo = mid;
      else hi = mid;
    }
    int rest = rank - count(lo + 1);
    // the rest-th item of level lo, sequences in order
    each(p, tpc, [&](const PromptLevels& v, int s0) {
      const int mine = above(v, lo) - above(v, lo + 1);
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += u;
      }
      const int sum = __shfl_sync(kFull, incl, 31);
      if (rest >= sum) {
        rest -= sum;
        return true;
      }
      const int who = __ffs(__ballot_sync(kFull, incl > rest)) - 1;
      const int before = __shfl_sync(kFull, incl - mine, who);
      const int at = __shfl_sync(kFull, v.lo, who);
      seq = s0 + who;
      tile = causal ? lo - at : rest - before;
      return false;
    });
    return true;
  }
};

// SHARED: the CTA is one of p.split that share an item, its only one.
template <int D, int G, bool SHARED>
__global__ void __launch_bounds__(kPrThreads, 1)
prompt_attention_kernel(const __grid_constant__ CUtensorMap tmap_q,
                        const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_v, const PromptArgs p) {
  using C = PromptCfg<D>;
  constexpr int kHeads = C::kHeads, kPairs = C::kPairs;
  constexpr int TPT = kPrRows / G;        // tokens of a Q tile
  constexpr int TPC = TPT * kPrTiles;     // tokens of an item
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + C::kBarOff;
  PromptItem* slots = reinterpret_cast<PromptItem*>(smem + C::kItemOff);
  volatile int* misc = reinterpret_cast<volatile int*>(smem + C::kMiscOff);
  volatile int* abort_flag = misc + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == kPrLoadWarp && lane == 0) {
    auto init = [&](int b, int count, int n) {
      for (int i = 0; i < n; ++i) mbar_init(bars + 8 * (b + i), count);
    };
    init(C::kHeadFull, 1, kHeads);
    init(C::kHeadFree, 1, kHeads);
    init(C::kPairLand, 1, kPairs);
    init(C::kPairFree, 1, kPairs);
    init(C::kSFull, 1, kPrTiles);
    for (int t = 0; t < kPrTiles; ++t) {
      init(C::kPFull + 2 * t, 5, 1);      // softmax warps, and the operands
      init(C::kPFull + 2 * t + 1, 4, 1);
    }
    init(C::kODone, 1, kPrTiles);
    init(C::kItem, 1, kPrSlots);
    init(C::kItemFree, 3 + 4 * kPrTiles, kPrSlots);  // copies, MMA, scrub, softmax warps
    init(C::kDrain, 1, 1);
    fence_barrier_init();
    *abort_flag = 0;
    slots[0].seq = -1;  // a shared item's end reads it even if a wait ran out
    tma_prefetch_desc(&tmap_q);
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
  }
  if (warp == kPrMmaWarp) {
    tmem_alloc(sbase + C::kMiscOff, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uint32_t(misc[0]);
  griddep_wait();  // what follows reads what kernels before may have written
  griddep_launch_dependents();

  // Key tiles of row tile t (0: it has no rows), those of them that are this
  // CTA's, and the first key tile that some row does not see whole.
  auto all_tiles = [&](const PromptItem& it, int t) {
    const int first = it.t0 + t * TPT, last = min(it.n, first + TPT);
    const int end = p.causal ? it.keys - it.n + last : it.keys;
    return first < it.n ? (end + kPrKeys - 1) / kPrKeys : 0;
  };
  auto tiles_of = [&](const PromptItem& it, int t) {
    return SHARED ? max(0, min(all_tiles(it, t), it.j1) - it.j0) : all_tiles(it, t);
  };
  auto first_tile = [&](const PromptItem& it) { return SHARED ? it.j0 : 0; };
  auto cut_of = [&](const PromptItem& it) {
    return p.causal ? (it.keys - it.n + it.t0 + 1) / kPrKeys : it.keys / kPrKeys;
  };
  // A role's next item from its slot (i counts items).
  auto take = [&](int i, PromptItem& it) {
    const int sl = i % kPrSlots;
    if (!pr_wait(bars + 8 * (C::kItem + sl), (i / kPrSlots) & 1, abort_flag)) return false;
    it = slots[sl];
    return true;
  };
  auto give_back = [&](int i) { mbar_arrive(bars + 8 * (C::kItemFree + i % kPrSlots)); };
  // Whole-warp wait.
  auto all_wait = [&](int bar, uint32_t parity) {
    return __all_sync(0xffffffffu, pr_wait(bars + 8 * bar, parity, abort_flag));
  };
  // Heads and pairs are numbered through the launch: number c of a ring of n is
  // the (c / n)-th in slot c % n.

  if (warp >= kPrLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPrRegsOther));
  if (warp == kPrLoadWarp) {
    // ================= copies (one thread) =================
    if (lane == 0) {
      uint32_t hc = 0, pc = 0;  // heads and pairs issued
      bool ok = true;
      for (int i = 0; ok; ++i) {
        PromptItem it;
        ok = take(i, it);
        if (!ok || it.seq < 0) break;
        give_back(i);
        const int ntiles = max(tiles_of(it, 0), tiles_of(it, 1));
        if (SHARED && ntiles == 0) continue;
        it.row0 += first_tile(it) * kPrKeys;
        auto rows = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, int head, int row) {
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(dst + h * C::kHalf, map, bar, h * 64, head, row);
        };
        const uint32_t hb = hc % kHeads;
        ok = hc < kHeads || pr_wait(bars + 8 * (C::kHeadFree + hb), (hc / kHeads - 1) & 1, abort_flag);
        if (!ok) break;
        const uint32_t hfull = bars + 8 * (C::kHeadFull + hb), head = sbase + hb * C::kHeadTile;
        mbar_arrive_expect_tx(hfull, C::kHeadTile);
#pragma unroll
        for (int t = 0; t < kPrTiles; ++t)
          rows(head + t * C::kTile, &tmap_q, hfull, it.kvh * G, it.qs + it.t0 + t * TPT);
        rows(head + kPrTiles * C::kTile, &tmap_k, hfull, it.kvh, it.row0);
        ++hc;
        for (int j = 0; j < ntiles; ++j) {
          const uint32_t st = pc % kPairs;
          ok = pc < kPairs || pr_wait(bars + 8 * (C::kPairFree + st), (pc / kPairs - 1) & 1, abort_flag);
          if (!ok) break;
          const bool more = j + 1 < ntiles;
          const uint32_t bar = bars + 8 * (C::kPairLand + st);
          const uint32_t pair = sbase + C::kPairOff + st * C::kPairTile;
          mbar_arrive_expect_tx(bar, more ? C::kPairTile : C::kTile);
          rows(pair, &tmap_v, bar, it.kvh, it.row0 + j * kPrKeys);
          if (more) rows(pair + C::kTile, &tmap_k, bar, it.kvh, it.row0 + (j + 1) * kPrKeys);
          ++pc;
        }
      }
      if (!ok) pr_abort(abort_flag);
      if (*abort_flag) {  // the copies in flight land before the CTA ends
        for (uint32_t c = hc > kHeads ? hc - kHeads : 0; c < hc; ++c)
          (void)mbar_wait_bounded(bars + 8 * (C::kHeadFull + c % kHeads), (c / kHeads) & 1);
        for (uint32_t c = pc > kPairs ? pc - kPairs : 0; c < pc; ++c)
          (void)mbar_wait_bounded(bars + 8 * (C::kPairLand + c % kPairs), (c / kPairs) & 1);
      }
    }
    __syncwarp();
  } else if (warp == kPrItemWarp) {
    // ===== the CTA's (cluster's) items: rounds of one per CTA, every other one from the
    // far end (whoever has the longest of one round gets the shortest of the next) =====
    if (blockIdx.x == 0)
      for (int s = lane; s < p.num_seqs; s += 32)
        if (prompt_seq(p, s).bad) atomicOr(&g_prompt_error, kErrBadQueryRange);
    // Sequences from the first on that ends before it begins are left out: the others'
    // rows lie behind one another, so that no two write one row, and their items are
    // no more than the launch took for granted (a cluster has one item).
    int seqs = p.num_seqs;
#pragma unroll 1
    for (int s = lane; s < p.num_seqs; s += 32)
      if (__ldg(p.q_start + s + 1) < __ldg(p.q_start + s)) seqs = min(seqs, s);
    seqs = __reduce_min_sync(0xffffffffu, seqs);
    bool ok = true;
    auto publish = [&](const auto& table) {
      bool more = true;
#pragma unroll 1
      for (int k = 0; ok && more; ++k) {
        const int split = SHARED ? p.split : 1;
        const long long g = gridDim.x / split, mine = blockIdx.x / split;
        const long long work = k * g + ((k & 1) ? g - 1 - mine : mine);
        const long long rank = work / p.kv_heads;
        PromptItem it = {-1, 0, 0, 0, 0, 0, 0, 0, 0, 0};
        int seq = -1, tile = 0;
        more = rank <= INT_MAX && table.item(p, TPC, int(rank), seq, tile);
        if (more) {
          const PromptSeq q = prompt_seq(p, seq);
          it.seq = seq;
          it.kvh = int(work - rank * p.kv_heads);
          it.qs = q.qs;
          it.n = q.n;
          it.keys = q.keys;
          it.t0 = tile * TPC;
          it.row0 = p.kv_lens ? seq * p.kv_stride : q.qs;
          const int tiles = max(all_tiles(it, 0), all_tiles(it, 1));
          const int part = blockIdx.x % split;
          it.j0 = int((long long)tiles * part / split);
          it.j1 = int((long long)tiles * (part + 1) / split);
        }
        const int sl = k % kPrSlots;
        ok = k < kPrSlots || all_wait(C::kItemFree + sl, (k / kPrSlots - 1) & 1);
        if (ok && lane == 0) {
          slots[sl] = it;
          mbar_arrive(bars + 8 * (C::kItem + sl));
        }
      }
    };
    if (p.num_seqs <= 32) {
      PromptTable<1> table;
      table.seqs = seqs;
      table.load(p, TPC);
      publish(table);
    } else {
      PromptTable<kPrRegSets> table;
      table.seqs = seqs;
      table.load(p, TPC);
      publish(table);
    }
    if (!ok && lane == 0) pr_abort(abort_flag);
  } else if (warp == kPrScrubWarp) {
    // ===== every tile's operands: V of those that the mask cuts loses the rows past the
    // sequence's end, NaN and infinities =====
    uint32_t pc = 0, tc[kPrTiles] = {0, 0};  // pairs; P tiles of row tile t
    bool ok = true;
    for (int i = 0; ok; ++i) {
      PromptItem it;
      ok = __all_sync(0xffffffffu, take(i, it));
      if (!ok || it.seq < 0) break;
      const int nt[kPrTiles] = {tiles_of(it, 0), tiles_of(it, 1)};
      const int ntiles = max(nt[0], nt[1]), cut = cut_of(it) - first_tile(it);
      for (int j = 0; ok && j < ntiles; ++j, ++pc) {
        const uint32_t st = pc % kPairs;
        ok = all_wait(C::kPairLand + st, (pc / kPairs) & 1);
        if (!ok) break;
        if (j >= cut) {
          // 16-byte chunks of the rows that are the sequence's; eight loads at a
          // time (one took 5300 cycles a tile, on short prompts' critical path)
          const int live = min(it.keys - (first_tile(it) + j) * kPrKeys, kPrKeys) * 8;
          bool found = false;
#pragma unroll 1
          for (int h = 0; h < D / 64; ++h) {
            const uint32_t v = sbase + C::kPairOff + st * C::kPairTile + h * C::kHalf;
            for (int x = live + lane; x < kPrKeys * 8; x += 32) st_shared_zero16(v + x * 16);
#pragma unroll 1
            for (int x0 = lane; x0 < live; x0 += 256) {
              uint32_t w[8][4], odd = 0;
#pragma unroll
              for (int u = 0; u < 8; ++u) {
                const int x = min(x0 + 32 * u, live - 1);
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[u][0]), "=r"(w[u][1]), "=r"(w[u][2]), "=r"(w[u][3])
                             : "r"(v + x * 16)
                             : "memory");
              }
#pragma unroll
              for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int c = 0; c < 4; ++c) odd |= nonfinite2(w[u][c]);
              if (odd & 0x80008000u) {
                found = true;
                for (int u = 0; u < 8; ++u) {
                  const int x = min(x0 + 32 * u, live - 1);
#pragma unroll
                  for (int c = 0; c < 4; ++c) {
                    uint32_t y;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(y) : "r"(v + x * 16 + c * 4) : "memory");
                    const uint32_t bad = (nonfinite2(y) & 0x80008000u) >> 15;
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(v + x * 16 + c * 4), "r"(y & ~(bad * 0xffffu))
                                 : "memory");
                  }
                }
              }
            }
          }
          fence_proxy_async_smem();
          if (__any_sync(0xffffffffu, found) && lane == 0)
            *const_cast<volatile int*>(&slots[i % kPrSlots].odd) = 1;
          __syncwarp();
        }
        // one arrival in each phase of the tiles' P: not before the last one's end
#pragma unroll
        for (int t = 0; t < kPrTiles; ++t) {
          if (j >= nt[t]) continue;
          ok = ok && (tc[t] == 0 || all_wait(C::kPFull + 2 * t, (tc[t] - 1) & 1));
          if (ok && lane == 0) mbar_arrive(bars + 8 * (C::kPFull + 2 * t));
          ++tc[t];
        }
      }
      __syncwarp();
      if (lane == 0) give_back(i);
    }
    if (!ok && lane == 0) pr_abort(abort_flag);
  } else if (warp == kPrMmaWarp) {
    // ================= MMA issue =================
    const uint32_t tmem = __shfl_sync(0xffffffffu, uint32_t(misc[0]), 0);
    // The warp runs as a whole and elects a lane for the MMAs, whose descriptors
    // are then values of the warp: from a branch on the lane number an MMA takes
    // longer to issue than to run (1 x 16384 tokens: 1784 us so, 1555 with the lane
    // elected).
    // Operands by their offset: in a cluster a shared address names its CTA above it.
    const uint32_t ops = sbase & 0x3ffffu;
    constexpr uint32_t kIdescS = idesc_bf16_f32(kPrRows, kPrKeys, 0, 0);
    constexpr uint32_t kIdescPV = idesc_bf16_f32(kPrRows, D, 0, 1);
    auto ready = [&](int bar, uint32_t parity) {
      if (!all_wait(bar, parity)) return false;
      tc_fence_after();
      return true;
    };
    auto commit = [&](int bar) {
      if (elect_lane()) umma_commit(bars + 8 * bar);
    };
    uint32_t hc = 0, pc = 0;         // heads and pairs consumed
    uint32_t tc[kPrTiles] = {0, 0};  // P tiles of row tile t
    bool ok = true;
    for (int i = 0; ok; ++i) {
      PromptItem it;
      ok = __all_sync(0xffffffffu, take(i, it));
      if (!ok || __shfl_sync(0xffffffffu, it.seq, 0) < 0) break;
      if (lane == 0) give_back(i);
      __syncwarp();
      const int nt[kPrTiles] = {__shfl_sync(0xffffffffu, tiles_of(it, 0), 0),
                                __shfl_sync(0xffffffffu, tiles_of(it, 1), 0)};
      const int ntiles = max(nt[0], nt[1]);
      if (SHARED && ntiles == 0) continue;
      const uint32_t hb = hc % kHeads;
      const uint32_t head = ops + hb * C::kHeadTile;
      auto issue_s = [&](int t, uint32_t k) {
        const uint32_t q = head + t * C::kTile;
        if (elect_lane()) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const uint32_t off = ((x >> 2) * C::kHalf + (x & 3) * 32) >> 4;
            umma_bf16(tmem + t * C::kTileCols, desc_at<16>((q >> 4) + off),
                      desc_at<16>((k >> 4) + off), kIdescS, x > 0);
          }
          umma_commit(bars + 8 * (C::kSFull + t));
        }
      };
      // keys [64 half, 64 half + 64) of a tile
      auto issue_pv = [&](int t, uint32_t v, int half, bool first) {
        const uint32_t at = tmem + t * C::kTileCols;
        if (elect_lane()) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int x = half * 4 + y;
            umma_bf16_ts(at + 128, at + 8 * x, desc_at<C::kHalf>((v >> 4) + x * 128), kIdescPV,
                         !first || x > 0);
          }
        }
      };
      ok = ready(C::kHeadFull + hb, (hc / kHeads) & 1);
      if (!ok) break;
      ++hc;
#pragma unroll
      for (int t = 0; t < kPrTiles; ++t)
        if (nt[t] > 0) issue_s(t, head + kPrTiles * C::kTile);
      if (ntiles == 1) commit(C::kHeadFree + hb);
#pragma unroll 1
      for (int j = 0; ok && j < ntiles; ++j, ++pc) {
        const uint32_t v = ops + C::kPairOff + (pc % kPairs) * C::kPairTile;
#pragma unroll
        for (int t = 0; t < kPrTiles; ++t) {
          if (!ok || j >= nt[t]) continue;
          ok = ready(C::kPFull + 2 * t, tc[t] & 1);
          if (!ok) continue;
          issue_pv(t, v, 0, j == 0);
          ok = ready(C::kPFull + 2 * t + 1, tc[t] & 1);
          if (!ok) continue;
          ++tc[t];
          issue_pv(t, v, 1, false);
          if (j + 1 < nt[t]) issue_s(t, v + C::kTile);
          else commit(C::kODone + t);
        }
        if (!ok) break;
        commit(C::kPairFree + pc % kPairs);
        if (j + 2 == ntiles) commit(C::kHeadFree + hb);
      }
    }
    if (!ok && lane == 0) pr_abort(abort_flag);
    __syncwarp();
    // every MMA is done before tensor memory is given back
    commit(C::kDrain);
    (void)mbar_wait_bounded(bars + 8 * C::kDrain, 0);
    __syncwarp();
  }
    if constexpr (SHARED) {
      __syncwarp();
      cluster_sync_all();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPrRegsSoftmax));
    // ================= softmax and output: warpgroup wg owns Q tile wg =================
    const int wg = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t at = tmem + wg * C::kTileCols + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t p_full = bars + 8 * (C::kPFull + 2 * wg);
    const bool neg = p.scale_log2 < 0.f;
    const float scale = fabsf(p.scale_log2);
    const uint64_t sc2 = f2_pack(scale, scale);
    uint32_t sc = 0, oc = 0;  // S tiles, items
    float m = -INFINITY, lsum = 0.f;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      PromptItem it;
      ok = __all_sync(0xffffffffu, take(i, it));
      if (!ok || it.seq < 0) break;
      const int tok = it.t0 + wg * TPT + r / G;
      const bool valid = tok < it.n;
      // rows past the end see what the last row does, and are not stored
      const int limit = p.causal ? it.keys - it.n + min(tok, it.n - 1) : it.keys - 1;
      const int tiles = tiles_of(it, wg);
      m = -INFINITY;
      lsum = 0.f;
      for (int j = 0; j < tiles; ++j, ++sc) {
        ok = all_wait(C::kSFull + wg, sc & 1);
        if (!ok) break;
        tc_fence_after();
        float s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(at + 32 * c, s[c]);
        tmem_wait_ld();
        if (neg) {
#pragma unroll
          for (int x = 0; x < 128; ++x) s[x >> 5][x & 31] = -s[x >> 5][x & 31];
        }
        const int last = limit - (first_tile(it) + j) * kPrKeys;  // keys up to here are visible
        if (last < kPrKeys - 1) {
#pragma unroll
          for (int x = 0; x < 128; ++x)
            s[x >> 5][x & 31] = x <= last ? s[x >> 5][x & 31] : -INFINITY;
        }
        // P = 2^(x - m): the first 64 keys' with m as it is, and then m is
        // looked at; where it has to rise (and for the first tile) all again.
        // A row's m depends on its own scores alone.
        bool settled = false, stays = false;
        uint32_t pk[32];
        uint64_t ls2[2], nm2, ts2 = sc2;
        if (j > 0) {
          nm2 = f2_pack(-m, -m);
          ls2[0] = ls2[1] = 0ull;
          float ex[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int u = 0; u < 32; ++u) {
            weights(s[u >> 4][(2 * u) & 31], s[u >> 4][((2 * u) & 31) + 1], sc2, nm2, ls2[u & 1], pk[u]);
            ex[u & 3] = max3f(ex[u & 3], s[2 + (u >> 4)][(2 * u) & 31], s[2 + (u >> 4)][((2 * u) & 31) + 1]);
          }
          const float mx = max3f(fmaxf(ex[0], ex[1]), ex[2], ex[3]) * scale;
          stays = fabsf(m) < kPrLarge && f2_sum(ls2) <= 65536.f && mx <= m + kPrMost;
          settled = __all_sync(0xffffffffu, stays);
        }
        if (!settled) {
          float ex[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int x = 0; x < 128; x += 2)
            ex[(x >> 1) & 3] = max3f(ex[(x >> 1) & 3], s[x >> 5][x & 31], s[x >> 5][(x & 31) + 1]);
          const float mx = max3f(fmaxf(ex[0], ex[1]), ex[2], ex[3]) * scale;
          const float m_new = stays ? m : fmaxf(m, mx);
          if (fabsf(m_new) >= kPrLarge) {  // scores rounded as the maximum is
#pragma unroll
            for (int x = 0; x < 128; x += 2)
              f2_unpack(f2_mul(f2_pack(s[x >> 5][x & 31], s[x >> 5][(x & 31) + 1]), sc2),
                        s[x >> 5][x & 31], s[x >> 5][(x & 31) + 1]);
            ts2 = f2_pack(1.f, 1.f);
          }
          if (j > 0) {
            const float alpha = m_new == m ? 1.f : ex2(m - m_new);
            const uint64_t al2 = f2_pack(alpha, alpha);
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              float o[16];
              tmem_ld16(at + 128 + c * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; x += 2)
                f2_unpack(f2_mul(f2_pack(o[x], o[x + 1]), al2), o[x], o[x + 1]);
              tmem_st16(at + 128 + c * 16, o);
            }
            lsum *= alpha;
          }
          m = m_new;
          // (no score above -inf yet: weights of 0)
          nm2 = f2_pack(m == -INFINITY ? 0.f : -m, m == -INFINITY ? 0.f : -m);
          ls2[0] = ls2[1] = 0ull;
#pragma unroll
          for (int u = 0; u < 32; ++u)
            weights(s[u >> 4][(2 * u) & 31], s[u >> 4][((2 * u) & 31) + 1], ts2, nm2, ls2[u & 1], pk[u]);
        }
        auto leave = [&](int half) {  // P of 64 keys, 32 columns
          tmem_st32u(at + 32 * half, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + 8 * half);
        };
        leave(0);
#pragma unroll
        for (int u = 0; u < 32; ++u)
          weights(s[2 + (u >> 4)][(2 * u) & 31], s[2 + (u >> 4)][((2 * u) & 31) + 1], ts2, nm2,
                  ls2[u & 1], pk[u]);
        leave(1);
        lsum += f2_sum(ls2);
      }
      if (!ok) break;
      if (tiles > 0) {
        ok = all_wait(C::kODone + wg, oc & 1);
        if (!ok) break;
        ++oc;
        tc_fence_after();
        const float inv = 1.f / lsum;
        const size_t row = size_t(it.qs + tok) * p.q_heads + size_t(it.kvh) * G + r % G;
        __nv_bfloat16* out = p.out + row * D;
        const bool odd = *const_cast<volatile int*>(&slots[i % kPrSlots].odd) != 0;
        const int cut = max(cut_of(it), first_tile(it));
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          if (SHARED && !odd) break;
          float o[32];
          tmem_ld32(at + 128 + c * 32, o);
          tmem_wait_ld();
          if (odd && valid) {
            // what was taken out of the cut tiles: an infinity or NaN of a
            // visible key makes the element that
            const __nv_bfloat16* v =
                p.v + (it.row0 + (long long)cut * kPrKeys) * p.v_stride + it.kvh * D + c * 32;
            const int end = SHARED ? min(limit, it.j1 * kPrKeys - 1) : limit;
            for (int key = cut * kPrKeys; key <= end; ++key, v += p.v_stride) {
#pragma unroll
              for (int x = 0; x < 32; ++x) {
                const float y = __bfloat162float(v[x]);
                if (!isfinite(y)) o[x] += y;
              }
            }
          }
          if (SHARED) {
            tmem_st32(at + 128 + c * 32, o);  // joined with the other CTAs' below
            tmem_wait_st();
          } else if (valid) {
#pragma unroll
            for (int x = 0; x < 32; x += 16)
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                               out + c * 32 + x),
                           "r"(pack_bf16x2(o[x] * inv, o[x + 1] * inv)),
                           "r"(pack_bf16x2(o[x + 2] * inv, o[x + 3] * inv)),
                           "r"(pack_bf16x2(o[x + 4] * inv, o[x + 5] * inv)),
                           "r"(pack_bf16x2(o[x + 6] * inv, o[x + 7] * inv)),
                           "r"(pack_bf16x2(o[x + 8] * inv, o[x + 9] * inv)),
                           "r"(pack_bf16x2(o[x + 10] * inv, o[x + 11] * inv)),
                           "r"(pack_bf16x2(o[x + 12] * inv, o[x + 13] * inv)),
                           "r"(pack_bf16x2(o[x + 14] * inv, o[x + 15] * inv))
                           : "memory");
          }
        }
      }
      tc_fence_before();  // the next item's P arrives after O was read
      __syncwarp();
      if (lane == 0) give_back(i);
    }
    if (!ok && lane == 0) pr_abort(abort_flag);
    if constexpr (SHARED) {
      // A shared item, the CTA's only one: its rows -- O, the maximum and the
      // sum -- over the rings once both row tiles are through with them.
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const int row = wg * kPrRows + r;
      float2* ml = reinterpret_cast<float2*>(smem + C::kJoinMl);
      const bool some = ok && oc > 0;  // this row tile had keys here
      ml[row] = some ? make_float2(m, lsum) : make_float2(-INFINITY, 0.f);
      if (some) {
        float4* dst = reinterpret_cast<float4*>(smem) + row * (D / 4);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32(at + 128 + c * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 8; ++x)  // rotated: a warp's rows stand in different banks
            dst[(c * 8 + x + lane) % (D / 4)] =
                make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        }
      }
      // (here, where the warps have their registers)
      const PromptItem it = slots[0];
      __syncwarp();
      cluster_sync_all();
      if (it.seq >= 0) {
        const int part = blockIdx.x % p.split, share = kPrTiles * kPrRows / p.split;
#pragma unroll 1
        for (int x = threadIdx.x; x < share * (D / 8); x += 256) {
          const int row = part * share + x / (D / 8), col = x % (D / 8);  // eight columns
          const int tok = it.t0 + row / G;
          if (tok >= it.n) continue;
          float2 ml[kPrMaxSplit];
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < kPrMaxSplit; ++c) {
            ml[c] = make_float2(-INFINITY, 0.f);
            if (c < p.split)
              ml[c] = cluster_ld<float2>(sbase + C::kJoinMl + row * 8, c);
            top = fmaxf(top, ml[c].x);
          }
          float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll
          for (int c = 0; c < kPrMaxSplit; ++c) {
            if (c >= p.split || ml[c].y == 0.f) continue;
            const float f = ex2(ml[c].x - top);
            sum += f * ml[c].y;
            const uint32_t base = sbase + row * (D * 4);
            const float4 a = cluster_ld<float4>(base + (2 * col + (row & 31)) % (D / 4) * 16, c);
            const float4 b = cluster_ld<float4>(base + (2 * col + 1 + (row & 31)) % (D / 4) * 16, c);
            o[0] += f * a.x;
            o[1] += f * a.y;
            o[2] += f * a.z;
            o[3] += f * a.w;
            o[4] += f * b.x;
            o[5] += f * b.y;
            o[6] += f * b.z;
            o[7] += f * b.w;
          }
          const float inv = 1.f / sum;
          *reinterpret_cast<uint4*>(p.out +
                                    (size_t(it.qs + tok) * p.q_heads + size_t(it.kvh) * G + row % G) * D +
                                    col * 8) =
              make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                         pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
        }
      }
      __syncwarp();
    }
  }

  if constexpr (SHARED) cluster_sync_all();  // no CTA leaves while another reads its memory
  tc_fence_before();
  __syncthreads();
  if (warp == kPrMmaWarp) tmem_dealloc(tmem, C::kTmemCols);
}

template <int D, int G, bool SHARED>
cudaError_t launch_prompt_t(const PromptArgs& a, long long ctas, const CUtensorMap* tq,
                            const CUtensorMap* tk, const CUtensorMap* tv, cudaStream_t stream) {
  using C = PromptCfg<D>;
  static std::atomic<int> attr_done[kAttrMaxDevices];
  cudaError_t e =
      set_smem_limit_once(prompt_attention_kernel<D, G, SHARED>, C::kSmemBytes, attr_done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kPrThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(a.split);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SHARED ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, prompt_attention_kernel<D, G, SHARED>, *tq, *tk, *tv, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <bool SHARED>
cudaError_t launch_prompt(const PromptArgs& a, int d_head, long long ctas, const CUtensorMap* tq,
                          const CUtensorMap* tk, const CUtensorMap* tv, cudaStream_t stream) {
  const int group = a.q_heads / a.kv_heads;
#define PKV_PROMPT_CASE(GG)                                                               \
  if (group == GG)                                                                        \
    return d_head == 128 ? launch_prompt_t<128, GG, SHARED>(a, ctas, tq, tk, tv, stream)  \
                         : launch_prompt_t<64, GG, SHARED>(a, ctas, tq, tk, tv, stream)
  PKV_PROMPT_CASE(1);
  PKV_PROMPT_CASE(2);
  PKV_PROMPT_CASE(4);
  PKV_PROMPT_CASE(8);
  PKV_PROMPT_CASE(16);
#undef PKV_PROMPT_CASE
  return cudaErrorInvalidValue;
}

}  // namespace pkv
