// Attention of whole prompts: packed sequences of different lengths, grouped
// heads, K and V as contiguous bf16 rows.
//
//   out[i] = softmax(q_i K^T scale) V  over keys 0 .. L - n + i  (all L keys
//   when not causal), i < n the sequence's queries, L its keys (n = L for a
//   prompt; the block-scaled prefill has a cached prefix before its queries).
//
// Two matrix products of 2 n L d flops each per head, half of that under the
// causal mask, over O((n + L) d) bytes: bound by the tensor cores.  Layout:
//  * an item is TILES (times two in a pair) tiles of 128 rows -- 128 / G tokens
//    times the G query heads of one KV head -- against the keys in tiles of
//    128.  S and O of a tile stand in tensor memory, P (bf16) is written over
//    S and read from there by the second product.
//  * d_head 128: TILES 2, and two CTAs form a pair (cta_group::2): one MMA
//    covers a row tile of each CTA, and each CTA holds half of the key tile's
//    K rows and V columns.  One CTA alone reads 8 KB of operands per 64-cycle
//    MMA from shared memory, all its bandwidth, while copies write there too.
//  * d_head 64: TILES 1 and two CTAs per SM, whose softmax and MMA phases
//    overlap, as do one's start and the other's work.
//  * a thread owns a row in the softmax: no shuffles.  The running maximum is
//    the ceiling of the largest score seen when it was last raised; a tile
//    keeps it while every row's sum of weights over 64 keys is at most 2^16,
//    so most tiles need no maximum.  It is a whole number, so raising it scales
//    by a power of two, which rounds neither P nor O.
//  * P in bf16 is off by 2^-8 of each weight at most, as the bf16 output is of
//    itself; S, O, the weights' sum and the maximum are float32.
//  * items are taken longest first over all sequences (each CTA works its item
//    out of q_start), heads side by side.
// Keys that no row sees: V rows past a sequence's end, which belong to the next
// one or nobody, are zeroed in shared memory; NaN and infinities of V in the
// tiles that the mask cuts are taken out of the product (0 times them is NaN)
// and added at the end to the rows that see them.
#include <algorithm>
#include <climits>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tcgen05.cuh"

namespace pkv {

static __device__ unsigned g_prompt_error = 0;

constexpr int kPrRows = 128;  // rows of a Q tile
constexpr int kPrKeys = 128;  // keys of a K / V tile
constexpr float kPrMaxSum = 65536.f;

template <int D, bool PAIR>
struct PromptCfg {
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int kTiles = D == 128 ? 2 : 1;  // Q tiles of a CTA
  static constexpr int kSoftWarps = 4 * kTiles;
  static constexpr int kThreads = kSoftWarps * 32 + 96;
  static constexpr int kLoadWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1,
                       kScrubWarp = kSoftWarps + 2;
  static constexpr int kQHalf = kPrRows * 128;             // 128 rows x 64 columns
  static constexpr int kQTile = (D / 64) * kQHalf;
  static constexpr int kKRows = kPrKeys / kCtas;           // K rows that this CTA holds
  static constexpr int kKHalf = kKRows * 128;
  static constexpr int kKTile = (D / 64) * kKHalf;
  static constexpr int kVHalf = kPrKeys * 128;
  static constexpr int kVCols = D / kCtas;                 // V columns that this CTA holds
  static constexpr int kVTile = (kVCols / 64) * kVHalf;
  static constexpr int kKStages = PAIR ? 5 : (D == 128 ? 2 : 3);
  static constexpr int kVStages = PAIR ? 5 : 2;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + kTiles * kQTile;
  static constexpr int kVOff = kKOff + kKStages * kKTile;
  static constexpr int kBarOff = kVOff + kVStages * kVTile;
  // barriers
  static constexpr int kQFull = 0, kKFull = 1, kKEmpty = kKFull + kKStages,
                       kVFull = kKEmpty + kKStages, kVEmpty = kVFull + kVStages,
                       kVLand = kVEmpty + kVStages, kVReady = kVLand + kVStages,
                       kSFull = kVReady + kVStages, kPFull = kSFull + 2, kODone = kPFull + 2,
                       kDrain = kODone + 2, kNumBars = kDrain + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;  // tmem, abort, non-finite, item (3)
  static constexpr int kSmemBytes = kMiscOff + 32 + 1024;
  static constexpr uint32_t kTmemCols = kTiles == 2 ? 512 : 256;
  static constexpr uint32_t kTileCols = 256;               // S / P, then O at 128
  static_assert(kTiles == 2 ? kSmemBytes <= 232448 : 2 * (kSmemBytes + 1024) <= 233472,
                "one CTA of two tiles, two CTAs of one, to an SM's shared memory");
};

// ---- cluster forms
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

template <bool PAIR>
struct Pr {
  static __device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    return PAIR ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
  }
  // Bounded; gives up as soon as another role of this CTA has aborted.
  static __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity,
                                              volatile int* abort_flag) {
    for (uint32_t i = 0; i < kWaitPollLimit; ++i) {
      if (try_wait(bar, parity)) return true;
      if ((i & 255u) == 255u && *abort_flag) return false;
    }
    return false;
  }
  static __device__ __forceinline__ void wait_anyway(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < kWaitPollLimit; ++i)
      if (try_wait(bar, parity)) return;
  }
  // One arrival on the leading CTA's barrier (`bar` as mapped there).
  static __device__ __forceinline__ void arrive(uint32_t bar) {
    if constexpr (PAIR) mbar_arrive_cluster(bar);
    else mbar_arrive(bar);
  }
  static __device__ __forceinline__ void load(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                              int c0, int c1, int c2) {
    if constexpr (PAIR)
      asm volatile(
          "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx"
          "::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
          "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
          : "memory");
    else
      tma_load_3d(dst, map, bar, c0, c1, c2);
  }
  static __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t acc) {
    if constexpr (PAIR)
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "setp.ne.b32 p, %4, 0;\n\t"
          "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
          "l"(a), "l"(b), "r"(idesc), "r"(acc)
          : "memory");
    else
      umma_bf16(d, a, b, idesc, acc);
  }
  static __device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                                uint32_t acc) {
    if constexpr (PAIR)
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "setp.ne.b32 p, %4, 0;\n\t"
          "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
          "r"(a), "l"(b), "r"(idesc), "r"(acc)
          : "memory");
    else
      umma_bf16_ts(d, a, b, idesc, acc);
  }
  // Arrives on `bar` in every CTA once the MMAs issued so far are done.
  static __device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (PAIR)
      asm volatile(
          "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
          " [%0], %1;" ::"r"(bar),
          "h"(uint16_t(3))
          : "memory");
    else
      umma_commit(bar);
  }
  static __device__ __forceinline__ void alloc(uint32_t dst, uint32_t cols) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst),
                   "r"(cols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(dst, cols);
      tmem_relinquish();
    }
  }
  static __device__ __forceinline__ void dealloc(uint32_t addr, uint32_t cols) {
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
                   : "memory");
    else
      tmem_dealloc(addr, cols);
  }
};

__device__ __forceinline__ void pr_abort(volatile int* abort_flag) {
  *abort_flag = 1;
  atomicOr(&g_prompt_error, kErrWaitTimeout);
}

// A sequence's rows and keys.
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

// Item `rank` of the launch, by one warp: items of `tpc` tokens, those with the
// most keys first.  The level of an item is its last key over tpc (all keys'
// when not causal); a sequence has one item of each of its levels, from
// lo = (keys - n) / tpc on.  Finds the level by bisection over the counts of
// items at or above one, then the sequence within it.  False: no such item.
__device__ __forceinline__ bool prompt_item(const PromptArgs& p, int tpc, long long rank, int& seq,
                                            int& tile) {
  const int lane = threadIdx.x & 31;
  constexpr unsigned kFull = 0xffffffffu;
  // items of sequence s at `level` or above
  auto above = [&](int s, int level) {
    const PromptSeq q = prompt_seq(p, s);
    const int items = (q.n + tpc - 1) / tpc;
    if (!p.causal) return q.keys / tpc >= level ? items : 0;
    const int lo = (q.keys - q.n) / tpc;
    return min(items, max(0, lo + items - level));
  };
  auto count = [&](int level) {
    long long c = 0;
    for (int s = lane; s < p.num_seqs; s += 32) c += above(s, level);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(kFull, c, o);
    return c;
  };
  int top = 0;
  for (int s = lane; s < p.num_seqs; s += 32) {
    const PromptSeq q = prompt_seq(p, s);
    if (q.n > 0) top = max(top, p.causal ? (q.keys - q.n) / tpc + (q.n + tpc - 1) / tpc : q.keys / tpc + 1);
  }
  top = __reduce_max_sync(kFull, top);  // no item at this level
  if (count(0) <= rank) return false;
  int lo = 0, hi = top;  // count(lo) > rank >= count(hi) = 0 or so
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (count(mid) > rank) lo = mid;
    else hi = mid;
  }
  long long rest = rank - (hi >= top ? 0 : count(hi));
  // the rest-th item of level lo, sequences in order
  for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
    const int s = s0 + lane;
    const int mine = s < p.num_seqs ? above(s, lo) - above(s, lo + 1) : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    const int all = __shfl_sync(kFull, incl, 31);
    if (rest < all) {
      const unsigned hit = __ballot_sync(kFull, incl > rest);
      const int who = __ffs(hit) - 1;
      const int before = __shfl_sync(kFull, incl - mine, who);
      seq = s0 + who;
      const PromptSeq q = prompt_seq(p, seq);
      tile = p.causal ? lo - (q.keys - q.n) / tpc : int(rest) - before;
      return true;
    }
    rest -= all;
  }
  return false;
}

template <int D, int G, bool PAIR>
__global__ void __launch_bounds__(PromptCfg<D, PAIR>::kThreads, PromptCfg<D, PAIR>::kTiles == 2 ? 1 : 2)
prompt_attention_kernel(const __grid_constant__ CUtensorMap tmap_q,
                        const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_v, const PromptArgs p) {
  using C = PromptCfg<D, PAIR>;
  using X = Pr<PAIR>;
  constexpr int kTiles = C::kTiles, kCtas = C::kCtas;
  constexpr int kKStages = C::kKStages, kVStages = C::kVStages;
  constexpr int TPT = kPrRows / G;              // tokens of a Q tile
  constexpr int TPS = TPT * kCtas;              // tokens that one MMA covers
  constexpr int TPC = TPS * kTiles;             // tokens of an item
  griddep_wait();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + C::kBarOff;
  volatile int* misc = reinterpret_cast<volatile int*>(smem + C::kMiscOff);
  volatile int* abort_flag = misc + 1;
  volatile int* nonfinite = misc + 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  const long long work = blockIdx.x / kCtas;
  const int kvh = int(work % p.kv_heads);
  if (work == 0 && rank == 0)
    for (int s = threadIdx.x; s < p.num_seqs; s += C::kThreads)
      if (prompt_seq(p, s).bad) atomicOr(&g_prompt_error, kErrBadQueryRange);

  // ---- this CTA's item, barriers, tensor memory
  if (warp == 0) {
    int seq = 0, tile = 0;
    const bool some = prompt_item(p, TPC, work / p.kv_heads, seq, tile);
    if (lane == 0) {
      misc[3] = some ? seq : -1;
      misc[4] = tile;
      *abort_flag = 0;
      *nonfinite = 0;
    }
  } else if (warp == C::kLoadWarp && lane == 0) {
    auto init = [&](int b, int n) { mbar_init(bars + 8 * b, n); };
    init(C::kQFull, 1);
    for (int s = 0; s < kKStages; ++s) {
      init(C::kKFull + s, 1);
      init(C::kKEmpty + s, 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      init(C::kVFull + s, 1);
      init(C::kVEmpty + s, 1);
      init(C::kVLand + s, 1);
      init(C::kVReady + s, kCtas);
    }
    for (int t = 0; t < 2; ++t) {
      init(C::kSFull + t, 1);
      init(C::kPFull + t, 4 * kCtas);
      init(C::kODone + t, 1);
    }
    init(C::kDrain, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tmap_q);
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
  }
  __syncthreads();
  const int seq = misc[3];
  if (seq < 0) return;  // both CTAs of a pair alike
  if (warp == C::kMmaWarp) X::alloc(sbase + C::kMiscOff, C::kTmemCols);
  tc_fence_before();
  if constexpr (PAIR) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uint32_t(misc[0]);
  const PromptSeq sq = prompt_seq(p, seq);
  const int t0 = misc[4] * TPC;
  const long long row0 = p.kv_lens ? (long long)seq * p.kv_stride : sq.qs;  // first K / V row
  // key tiles that each MMA row tile needs (0: it has no rows), and the first
  // key tile that some row does not see whole
  int nt[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int first = t0 + t * TPS, last = min(sq.n, first + TPS);
    const int end = p.causal ? sq.keys - sq.n + last : sq.keys;
    nt[t] = first < sq.n ? (end + kPrKeys - 1) / kPrKeys : 0;
  }
  const int ntiles = kTiles == 2 ? max(nt[0], nt[kTiles - 1]) : nt[0];
  const int cut = p.causal ? (sq.keys - sq.n + t0 + 1) / kPrKeys : sq.keys / kPrKeys;
  const uint32_t lead = PAIR ? in_cta(bars, 0) : bars;  // the leading CTA's barriers
  // the number of tile j among the cut tiles of its ring slot
  auto cut_phase = [&](int j) {
    const int st = j % kVStages;
    const int j0 = cut + (st - cut % kVStages + kVStages) % kVStages;
    return uint32_t((j - j0) / kVStages) & 1u;
  };

  if (warp == C::kLoadWarp) {
    // ================= copies (one thread) =================
    if (lane == 0) {
      int k_issued = 0, v_issued = 0;
      bool ok = true;
      if (rank == 0) mbar_arrive_expect_tx(bars + 8 * C::kQFull, kCtas * kTiles * C::kQTile);
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          X::load(sbase + C::kQOff + t * C::kQTile + h * C::kQHalf, &tmap_q, lead + 8 * C::kQFull,
                  h * 64, kvh * G, sq.qs + t0 + t * TPS + int(rank) * TPT);
      auto load_k = [&](int j) {
        const int st = j % kKStages;
        if (j >= kKStages && !X::wait(bars + 8 * (C::kKEmpty + st), (j / kKStages - 1) & 1, abort_flag))
          return false;
        if (rank == 0) mbar_arrive_expect_tx(bars + 8 * (C::kKFull + st), kCtas * C::kKTile);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          X::load(sbase + C::kKOff + st * C::kKTile + h * C::kKHalf, &tmap_k,
                  lead + 8 * (C::kKFull + st), h * 64, kvh,
                  int(row0) + j * kPrKeys + int(rank) * C::kKRows);
        ++k_issued;
        return true;
      };
      auto load_v = [&](int j) {
        const int st = j % kVStages;
        if (j >= kVStages && !X::wait(bars + 8 * (C::kVEmpty + st), (j / kVStages - 1) & 1, abort_flag))
          return false;
        // a cut tile lands on this CTA's own barrier, for the scrub warp
        const bool own = j >= cut;
        if (own) mbar_arrive_expect_tx(bars + 8 * (C::kVLand + st), C::kVTile);
        else if (rank == 0) mbar_arrive_expect_tx(bars + 8 * (C::kVFull + st), kCtas * C::kVTile);
        const uint32_t bar = own ? bars + 8 * (C::kVLand + st) : lead + 8 * (C::kVFull + st);
#pragma unroll
        for (int h = 0; h < C::kVCols / 64; ++h)
          X::load(sbase + C::kVOff + st * C::kVTile + h * C::kVHalf, &tmap_v, bar,
                  int(rank) * C::kVCols + h * 64, kvh, int(row0) + j * kPrKeys);
        ++v_issued;
        return true;
      };
      ok = load_k(0);
      for (int j = 0; ok && j < ntiles; ++j) {
        if (j + 1 < ntiles) ok = load_k(j + 1);
        ok = ok && load_v(j);
      }
      if (!ok) pr_abort(abort_flag);
      // after an abort: what this CTA can see of its copies lands before it ends
      if (*abort_flag) {
        if (rank == 0) {
          X::wait_anyway(bars + 8 * C::kQFull, 0);
          for (int j = max(0, k_issued - kKStages); j < k_issued; ++j)
            X::wait_anyway(bars + 8 * (C::kKFull + j % kKStages), (j / kKStages) & 1);
          for (int j = max(0, v_issued - kVStages); j < v_issued && j < cut; ++j)
            X::wait_anyway(bars + 8 * (C::kVFull + j % kVStages), (j / kVStages) & 1);
        }
        for (int j = max(cut, v_issued - kVStages); j < v_issued; ++j)
          X::wait_anyway(bars + 8 * (C::kVLand + j % kVStages), cut_phase(j));
      }
    }
    __syncwarp();
  } else if (warp == C::kScrubWarp) {
    // ===== V tiles that the mask cuts: rows past the end to zero, NaN and infinities out =====
    for (int j = cut; j < ntiles; ++j) {
      const int st = j % kVStages;
      const bool ok = __all_sync(0xffffffffu,
                                 X::wait(bars + 8 * (C::kVLand + st), cut_phase(j), abort_flag));
      if (!ok) {
        if (lane == 0) pr_abort(abort_flag);
        break;
      }
      const uint32_t v = sbase + C::kVOff + st * C::kVTile;
      const int live = sq.keys - j * kPrKeys;  // rows of this tile that are the sequence's
      bool found = false;
#pragma unroll 4
      for (int i = lane; i < C::kVTile / 16; i += 32) {
        const int row = (i >> 3) % kPrKeys;
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(v + i * 16)
                     : "memory");
        if (row >= live) {
          st_shared_zero16(v + i * 16);
          continue;
        }
        uint32_t odd = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) odd |= __vcmpgeu2(w[c] & 0x7fff7fffu, 0x7f807f80u);
        if (odd) {
          found = true;
#pragma unroll
          for (int c = 0; c < 4; ++c) w[c] &= ~__vcmpgeu2(w[c] & 0x7fff7fffu, 0x7f807f80u);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(v + i * 16), "r"(w[0]),
                       "r"(w[1]), "r"(w[2]), "r"(w[3])
                       : "memory");
        }
      }
      fence_proxy_async_smem();
      if (__any_sync(0xffffffffu, found) && lane == 0) {
#pragma unroll
        for (int c = 0; c < kCtas; ++c) {
          const uint32_t at = sbase + C::kMiscOff + 8;
          if constexpr (PAIR)
            asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(in_cta(at, c)), "r"(1) : "memory");
          else
            *nonfinite = 1;
        }
      }
      __syncwarp();
      if (lane == 0) X::arrive(lead + 8 * (C::kVReady + st));
    }
  } else if (warp == C::kMmaWarp) {
    // ================= MMA issue (one thread of the leading CTA) =================
    if (lane == 0 && rank == 0) {
      constexpr uint32_t kIdescS = idesc_bf16_f32(kPrRows * kCtas, kPrKeys, 0, 0);
      constexpr uint32_t kIdescPV = idesc_bf16_f32(kPrRows * kCtas, D, 0, 1);
      auto issue_s = [&](int t, int j) {
        const uint32_t q = sbase + C::kQOff + t * C::kQTile;
        const uint32_t k = sbase + C::kKOff + (j % kKStages) * C::kKTile;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          X::mma(tmem + t * C::kTileCols,
                 smem_desc_sw128(q + (i >> 2) * C::kQHalf + (i & 3) * 32, 16, 1024),
                 smem_desc_sw128(k + (i >> 2) * C::kKHalf + (i & 3) * 32, 16, 1024), kIdescS, i > 0);
        X::commit(bars + 8 * (C::kSFull + t));
      };
      auto issue_pv = [&](int t, int j) {
        const uint32_t v = sbase + C::kVOff + (j % kVStages) * C::kVTile;
        const uint32_t at = tmem + t * C::kTileCols;
#pragma unroll
        for (int i = 0; i < kPrKeys / 16; ++i)
          X::mma_ts(at + 128, at + 64 * (i >> 2) + 8 * (i & 3),
                    smem_desc_sw128(v + i * 2048, C::kVHalf, 1024), kIdescPV, j > 0 || i > 0);
        X::commit(bars + 8 * (C::kODone + t));
      };
      auto ready = [&](int bar, uint32_t parity) {
        if (!X::wait(bars + 8 * bar, parity, abort_flag)) return false;
        tc_fence_after();
        return true;
      };
      auto k_ready = [&](int j) { return ready(C::kKFull + j % kKStages, (j / kKStages) & 1); };
      auto v_ready = [&](int j) {
        return j < cut ? ready(C::kVFull + j % kVStages, (j / kVStages) & 1)
                       : ready(C::kVReady + j % kVStages, cut_phase(j));
      };
      bool ok = ready(C::kQFull, 0) && k_ready(0);
      if (ok) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
          if (nt[t] > 0) issue_s(t, 0);
        X::commit(bars + 8 * C::kKEmpty);
      }
      for (int j = 0; ok && j < ntiles; ++j) {
        ok = v_ready(j) && (j + 1 >= ntiles || k_ready(j + 1));
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (!ok || j >= nt[t]) continue;
          ok = ready(C::kPFull + t, j & 1);
          if (!ok) continue;
          issue_pv(t, j);
          if (t == kTiles - 1) X::commit(bars + 8 * (C::kVEmpty + j % kVStages));
          if (j + 1 < nt[t]) issue_s(t, j + 1);
        }
        if (!ok) break;
        // the last row tile has none of this tile: its slot is free all the same
        if (j >= nt[kTiles - 1]) X::commit(bars + 8 * (C::kVEmpty + j % kVStages));
        if (j + 1 < ntiles) X::commit(bars + 8 * (C::kKEmpty + (j + 1) % kKStages));
      }
      if (!ok) pr_abort(abort_flag);
      // every MMA is done before tensor memory is given back
      X::commit(bars + 8 * C::kDrain);
      X::wait_anyway(bars + 8 * C::kDrain, 0);
    }
    __syncwarp();
  } else {
    // ================= softmax and output: warpgroup wg owns Q tile wg =================
    const int wg = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int tok = t0 + wg * TPS + int(rank) * TPT + r / G;
    const bool valid = tok < sq.n;
    // rows past the end see what the last row does, and are not stored
    const int limit = p.causal ? sq.keys - sq.n + min(tok, sq.n - 1) : sq.keys - 1;
    const uint32_t at = tmem + wg * C::kTileCols + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t s_full = bars + 8 * (C::kSFull + wg), o_done = bars + 8 * (C::kODone + wg);
    const uint32_t p_full = lead + 8 * (C::kPFull + wg);
    const int tiles = nt[wg];
    const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
    float m = -INFINITY, lsum = 0.f;
    bool ok = true;
    for (int j = 0; j < tiles; ++j) {
      ok = __all_sync(0xffffffffu, X::wait(s_full, j & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const int key0 = j * kPrKeys;
      if (j == 0) {  // key 0 is visible to every row
        float va[32];
        tmem_ld32(at, va);
        tmem_wait_ld();
        float ex[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i <= limit) ex[i & 3] = fmaxf(ex[i & 3], va[i] * p.scale_log2);
        m = ceilf(fmaxf(fmaxf(ex[0], ex[1]), fmaxf(ex[2], ex[3])));
      }
#pragma unroll 1
      for (int g = 0; g < 2; ++g) {  // 64 keys at a time
        float va[32], vb[32];
        tmem_ld32(at + 64 * g, va);
        tmem_ld32(at + 64 * g + 32, vb);
        tmem_wait_ld();
        const int last = limit - key0 - 64 * g;  // keys of the group up to here are visible
        for (int attempt = 0;; ++attempt) {
          uint32_t pk[32];
          const uint64_t nm2 = f2_pack(-m, -m);
          uint64_t ls2[2] = {0ull, 0ull};
          if (last >= 63) {
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              const int kk = 2 * u;
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(kk < 32 ? va[kk] : vb[kk - 32], kk < 32 ? va[kk + 1] : vb[kk - 31]),
                               sc2, nm2), x0, x1);
              const float e0 = ex2(x0), e1 = ex2(x1);
              ls2[u & 1] = f2_add(ls2[u & 1], f2_pack(e0, e1));
              pk[u] = pack_bf16x2(e0, e1);
            }
          } else {
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              const int kk = 2 * u;
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(kk < 32 ? va[kk] : vb[kk - 32], kk < 32 ? va[kk + 1] : vb[kk - 31]),
                               sc2, nm2), x0, x1);
              const float e0 = kk <= last ? ex2(x0) : 0.f, e1 = kk + 1 <= last ? ex2(x1) : 0.f;
              ls2[u & 1] = f2_add(ls2[u & 1], f2_pack(e0, e1));
              pk[u] = pack_bf16x2(e0, e1);
            }
          }
          float a0, a1, b0, b1;
          f2_unpack(ls2[0], a0, a1);
          f2_unpack(ls2[1], b0, b1);
          const float sum = (a0 + a1) + (b0 + b1);
          // no weight is above the sum; NaN and infinity fail the test
          if (attempt > 0 || __all_sync(0xffffffffu, sum <= kPrMaxSum)) {
            lsum += sum;
            tmem_st32u(at + 64 * g, pk);
            break;
          }
          // raise the maximum to this group's
          float ex[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (i <= last) ex[i & 3] = fmaxf(ex[i & 3], va[i] * p.scale_log2);
            if (i + 32 <= last) ex[i & 3] = fmaxf(ex[i & 3], vb[i] * p.scale_log2);
          }
          const float m_new =
              fmaxf(m, ceilf(fmaxf(fmaxf(ex[0], ex[1]), fmaxf(ex[2], ex[3]))));
          const float alpha = m_new == m ? 1.f : ex2(m - m_new);
          if (j > 0) {  // after the product of the tile before
            ok = __all_sync(0xffffffffu, X::wait(o_done, (j - 1) & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const uint64_t al2 = f2_pack(alpha, alpha);
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              float o[16];
              tmem_ld16(at + 128 + c * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; i += 2)
                f2_unpack(f2_mul(f2_pack(o[i], o[i + 1]), al2), o[i], o[i + 1]);
              tmem_st16(at + 128 + c * 16, o);
            }
          }
          if (g == 1) {  // the first group's P, by an exact power of two
            tmem_wait_st();
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              float ph[16];
              tmem_ld16(at + 16 * c, ph);
              tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 16; ++u) {
                const uint32_t w = __float_as_uint(ph[u]);
                ph[u] = __uint_as_float(
                    pack_bf16x2(bf16_lo_to_f32(w) * alpha, bf16_hi_to_f32(w) * alpha));
              }
              tmem_st16(at + 16 * c, ph);
            }
          }
          lsum *= alpha;
          m = m_new;
        }
        if (!ok) break;
      }
      if (!ok) break;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) X::arrive(p_full);
    }
    if (ok && tiles > 0) {
      ok = __all_sync(0xffffffffu, X::wait(o_done, (tiles - 1) & 1, abort_flag));
      if (ok) {
        tc_fence_after();
        const float inv = 1.f / lsum;
        const size_t row = size_t(sq.qs + tok) * p.q_heads + size_t(kvh) * G + r % G;
        __nv_bfloat16* out = p.out + row * D;
        const bool odd = *nonfinite != 0;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32(at + 128 + c * 32, o);
          tmem_wait_ld();
          if (odd && valid) {
            // what was taken out of the cut tiles: an infinity or NaN of a
            // visible key makes the element that
            const __nv_bfloat16* v =
                p.v + (row0 + (long long)cut * kPrKeys) * p.v_stride + kvh * D + c * 32;
            for (int key = cut * kPrKeys; key <= limit; ++key, v += p.v_stride) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float x = __bfloat162float(v[i]);
                if (!isfinite(x)) o[i] += x;
              }
            }
          }
          if (valid) {
#pragma unroll
            for (int i = 0; i < 32; i += 16)
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                               out + c * 32 + i),
                           "r"(pack_bf16x2(o[i] * inv, o[i + 1] * inv)),
                           "r"(pack_bf16x2(o[i + 2] * inv, o[i + 3] * inv)),
                           "r"(pack_bf16x2(o[i + 4] * inv, o[i + 5] * inv)),
                           "r"(pack_bf16x2(o[i + 6] * inv, o[i + 7] * inv)),
                           "r"(pack_bf16x2(o[i + 8] * inv, o[i + 9] * inv)),
                           "r"(pack_bf16x2(o[i + 10] * inv, o[i + 11] * inv)),
                           "r"(pack_bf16x2(o[i + 12] * inv, o[i + 13] * inv)),
                           "r"(pack_bf16x2(o[i + 14] * inv, o[i + 15] * inv))
                           : "memory");
          }
        }
      }
    }
    if (!ok && lane == 0) pr_abort(abort_flag);
  }

  tc_fence_before();
  if constexpr (PAIR) cluster_sync_all();
  else __syncthreads();
  if (warp == C::kMmaWarp) X::dealloc(tmem, C::kTmemCols);
}

namespace {

template <int D, int G, bool PAIR>
cudaError_t launch_prompt_t(const PromptArgs& a, const CUtensorMap* tq, const CUtensorMap* tk,
                            const CUtensorMap* tv, cudaStream_t stream) {
  using C = PromptCfg<D, PAIR>;
  static std::atomic<int> attr_done[kAttrMaxDevices];
  cudaError_t e = set_smem_limit_once(prompt_attention_kernel<D, G, PAIR>, C::kSmemBytes, attr_done);
  if (e != cudaSuccess) return e;
  const int tpc = kPrRows / G * C::kCtas * C::kTiles;
  const long long grid = (a.total_q / tpc + (long long)a.num_seqs) * a.kv_heads * C::kCtas;
  if (grid > INT_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C::kCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, prompt_attention_kernel<D, G, PAIR>, *tq, *tk, *tv, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

int prompt_key_rows(int d_head) {
  return d_head == 128 ? PromptCfg<128, true>::kKRows : PromptCfg<64, false>::kKRows;
}
int prompt_value_rows() { return kPrKeys; }
int prompt_tile_rows() { return kPrRows; }

cudaError_t launch_prompt_attention(const PromptArgs& a, int d_head, const CUtensorMap* tq,
                                    const CUtensorMap* tk, const CUtensorMap* tv,
                                    cudaStream_t stream) {
  const int group = a.q_heads / a.kv_heads;
#define PKV_PROMPT_CASE(GG)                                                        \
  if (group == GG)                                                                 \
    return d_head == 128 ? launch_prompt_t<128, GG, true>(a, tq, tk, tv, stream)   \
                         : launch_prompt_t<64, GG, false>(a, tq, tk, tv, stream)
  PKV_PROMPT_CASE(1);
  PKV_PROMPT_CASE(2);
  PKV_PROMPT_CASE(4);
  PKV_PROMPT_CASE(8);
  PKV_PROMPT_CASE(16);
#undef PKV_PROMPT_CASE
  return cudaErrorInvalidValue;
}

// Device address of this unit's error word on the current device.
cudaError_t prompt_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_prompt_error);
}

unsigned read_prompt_error(bool clear) {
  unsigned word = 0;
  if (cudaMemcpyFromSymbol(&word, g_prompt_error, sizeof(word)) != cudaSuccess) return ~0u;
  if (clear) {
    const unsigned zero = 0;
    if (cudaMemcpyToSymbol(g_prompt_error, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  }
  return word;
}

}  // namespace pkv
