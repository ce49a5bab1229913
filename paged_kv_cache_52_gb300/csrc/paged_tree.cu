// Attention of trees of drafted tokens over the paged KV cache: the
// verification step of speculative decoding when the draft branches, on the
// 5th-generation tensor cores (tcgen05 + tensor memory).
//
// What is computed: sequence s has L = context_len cached positions, of which
// the last n <= 64 are the nodes of its tree.  Node t with ancestor mask M_t
// attends the committed keys j < L - n and the nodes u with bit u of M_t:
//   out[t, h] = sum_j p_j v_j,  p = softmax_j(scale q[t, h] . k_j)
// (the prefill's softmax(q K^T scale + mask) V with a tree in place of the
// causal triangle), GQA head h reading KV head h / G.  A row that sees no key
// is zero.
//
// Design (GB300):
//  * rows of a (sequence, KV head) pair are its n x G (node, head) rows,
//    node-major, in tiles of 128 = the MMA's M; every K/V byte is read once
//    for a tile pair.  The keys stream by in tiles of 128 (8 pages).
//  * the work is cut by key tiles, not by sequences: the tiles of all items
//    (pair, row group) laid end to end are divided evenly over one CTA per
//    SM, so a batch of ragged contexts, or one long one, loads every SM
//    alike.  An item that lies in one CTA is finished there, the pieces of a
//    cut item (at most two per CTA) go through the workspace and a merge
//    kernel by log-sum-exp.
//  * TILES = 1 (at most 128 rows a pair): the two softmax warpgroups take the
//    key tiles in turn, each with its own running max, sum and tensor-memory
//    accumulator; at the end of an item each row's two halves are combined,
//    both warpgroups reading both accumulators (half the columns each).
//    TILES = 2: warpgroup t owns row tile t and K/V tiles serve both.
//  * warps 0-3 and 4-7 softmax, correction and epilogue (thread = row =
//    tensor-memory lane), warp 8 loads K, 9 loads Q, works out the pieces and
//    issues Q K^T, 10 loads V, 11 issues P V.  The rings run on across items;
//    only Q and the accumulators change hands at an item's end.
//  * S = Q K^T lands in tensor memory, the softmax overwrites it with P as
//    bf16 hi + lo (two MMAs a step, an error of 2^-16 at most: a row may see very few
//    keys, where P rounded to one bf16 would move the output by 2^-8), and
//    P V reads P from tensor memory.
//  * only tiles that reach the tree apply a mask: 128 bits a row, made from
//    the 64-bit ancestor mask.  A masked key's P is 0, but 0 * NaN is not:
//    in those tiles every non-finite element of V is replaced by 0 in shared
//    memory and added, in the epilogue, to just the rows that see its node,
//    so a sibling's (or a stale row's) NaN or infinity reaches nobody else.
//  * every wait is bounded; a timeout sets the error word and an abort flag,
//    copies and MMAs in flight are drained and tensor memory is freed.
//
// What bounds it (us in a graph at 2070 MHz, 64 query and 8 KV heads of 128 unless
// said; shares from the profiler's counters):
//  * 16 x 4096, 16 nodes: 51.  HBM in the middle (64 KB per SM in 2730 cycles =
//    7 TB/s), 58% of its peak over the kernel; 31 us are the bytes.  The rest are
//    the ends: 2.3 until the first pages are asked for, 3 until they are there,
//    pieces that meet in a CTA (2-3 each), 4.5 for the merge.
//  * 64 x 8192, 64 nodes (two row tiles): 850-875, the tensor cores' 585 with P as
//    hi + lo.  5500 cycles a key tile for both row tiles, of which the tensor
//    pipe is busy for 56%: a row tile's chain of scores, softmax and products
//    (the softmax's two halves 1300 cycles each).
//  * 2 x 131072, 27 nodes, 32 query heads of 64: 107-111 (120 in some processes) of
//    79 for the bytes.  HBM runs at 63% of its peak and the tensor pipe is busy for
//    43% of the cycles, 770 of 1780 a tile: neither is full, and which wait of
//    the chain fills the rest has not been shown.
//  * 1 x 500, 8 nodes: 11.8, all latency: 1.3 for the split, 1.7 to the first
//    page, 2.7 for one tile of each warpgroup, 2.5 for its end, 0.8 + 2.4 for
//    the merge.
//  * a bound above the trees: with max_q_len x group > 128 every tree takes two row
//    tiles, also where the second has no rows.  max_q_len 64 instead of the trees' own:
//    16 x 4096, 16 nodes 65.7 against 50.7, 64 x 700, 4 nodes 57.8 / 44.5, 2 x 131072 161 / 108.
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tcgen05.cuh"

namespace pkv {

static __device__ unsigned g_tree_error = 0;

constexpr int kTrRows = 128;     // rows (node x head) per tile
constexpr int kTrKeys = 128;     // keys per K/V tile (8 pages)
constexpr int kTrThreads = 384;
constexpr int kTrRegsSoftmax = 192, kTrRegsIssue = 120;
constexpr int kTrKWarp = 8, kTrSWarp = 9, kTrVWarp = 10;  // 11 issues P V
constexpr uint32_t kTrTmemCols = 512;
constexpr float kTrRescale = 8.0f;     // log2 units: move the running max when it grows by > x256
// The most that a row's weights over 64 keys may add up to against the running max it
// has.  The accumulator holds weights times V, at most (L / 64 + 1) 2^24 max|V|: finite V
// up to 2^110 / (L + 64) cannot overflow it.  us with 2^16 / 2^24 / 2^64: 64 x 8192, 64
// nodes 885 / 873 / 874, 6 x 9000, 64 nodes, heads of 64 48.7 / 46.1 / 46.1, 16 x 4096, 16
// nodes 51.5 / 51.1 / 51.2.
constexpr float kTrMaxSum = 16777216.f;
constexpr int kTrMaxStages = 4;
// The fewest key tiles worth a piece: one for each softmax warpgroup (us with 2 / 1:
// three tiles, 1 x 384, 8 nodes 11.6 / 11.8; 1 x 2000, 16 nodes 15.4 either way).
constexpr int kTrMinTiles = 2;
// Key tiles' time that a second piece costs a CTA: the first one's end and the
// next one's start.  us with 1 / 2 / 3: 8 x 2000, 8 nodes 23.7 / 22.5 / 22.1, 64 x 700,
// 4 nodes 44.8 / 44.5 / 44.0, 32 x 1000, 16 nodes 37.6 / 36.4 / 36.1, 16 x 4096, 16
// nodes 50.8 / 50.7 / 49.8, 1 x 2000, 16 nodes 15.4 / 15.4 / 16.1, 2 x 131072, 27 nodes,
// heads of 64 106.7 / 107.3 / 108.3.
constexpr int kTrSlack = 2;
constexpr int kTrPieces = 5;  // piece descriptions in shared memory

template <int D, int TILES>
struct TreeSmem {
  // S, P and P V of a tile of heads of 128 go in two halves of 64 keys, so that
  // the products of one half and the next scores run while the other half is
  // weighed; heads of 64, with a third buffer, keep them whole.  us in halves / whole:
  // 64 x 8192, 64 nodes 856 / 941, 16 x 4096, 16 nodes 50.7 / 52.1, 64 x 700, 4 nodes
  // 44.5 / 47.6; heads of 64, 2 x 131072, 27 nodes 114.7 / 107.3.
  static constexpr int kParts = D == 128 ? 2 : 1;
  // Tensor memory: S/P buffers that the products take in turn, and the
  // warpgroups' accumulators.  Heads of 128: a buffer and an accumulator of 128
  // columns a warpgroup.  Heads of 64 leave room for a third buffer, so that a
  // warpgroup's next scores are made while its last P is still being multiplied.
  static constexpr int kBufs = D == 64 ? 3 : 2;
  static __device__ __forceinline__ uint32_t buf_col(int b) { return (D == 64 ? 128 : 256) * b; }
  static __device__ __forceinline__ uint32_t out_col(int w) {
    return D == 64 ? 384 + 64 * w : 256 * w + 128;
  }
  static constexpr int kHalf = 128 * 128;  // 128 rows x 64 bf16
  static constexpr int kTileBytes = (D / 64) * kHalf;
  static constexpr int kQBytes = TILES * kTileBytes;
  // Ring stages: what 227 KB hold beside Q.  A V tile also waits for its
  // softmax, a K tile only for its product.
  static constexpr int kKStages = D == 64 ? 4 : 3;
  static constexpr int kVStages = D == 64 ? 4 : (TILES == 1 ? 3 : 2);
  static constexpr int kKOff = kQBytes;
  static constexpr int kVOff = kKOff + kKStages * kTileBytes;
  static constexpr int kXchOff = kVOff + kVStages * kTileBytes;  // [2][128] (max, sum)
  static constexpr int kBarOff = kXchOff + 2 * kTrRows * 8;
  static constexpr int kNumBars = 2 + 4 * kTrMaxStages + 18 + 3 + kTrPieces;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  // tensor-memory base, abort flag; non-finite nodes [2] (64 bit); scan [12];
  // the start of the range; the pieces
  static constexpr int kPieceOff = kMiscOff + 16 + 16 + 48 + 48;
  static constexpr int kSmemBytes = kPieceOff + kTrPieces * 32;
  static_assert(kSmemBytes <= 232448, "tree tile does not fit in shared memory");
  static_assert(kKStages <= kTrMaxStages && kVStages <= kTrMaxStages, "ring stages");
  // a V slot's tile before is of a job at least kBufs back (the softmax's wait for V)
  static_assert(kVStages * TILES >= kBufs, "V stages");
};

enum TrBar {
  kTrQFull = 0, kTrQEmpty = 1,
  kTrKFull = 2, kTrKEmpty = kTrKFull + kTrMaxStages,
  kTrVFull = kTrKEmpty + kTrMaxStages, kTrVEmpty = kTrVFull + kTrMaxStages,
  // by half of the tile's keys and buffer: 3 h + b
  kTrSFull = kTrVEmpty + kTrMaxStages, kTrPFull = kTrSFull + 6, kTrDone = kTrPFull + 6,
  kTrXch = kTrDone + 6, kTrEpi = kTrXch + 1, kTrDrain = kTrEpi + 1, kTrPiece0 = kTrDrain + 1
};

// Where a CTA's range starts, for the merge: sequence (-1: no work), item of
// the sequence, first key tile, and the sequence's first row, nodes and row
// groups.
struct __align__(16) TreeStart {
  int seq, item, tile, qs, n, groups, pad[2];
};

struct TreeParams {
  const int32_t* q_start;
  const unsigned long long* tree_mask;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const void* v_pool;
  void* out;
  int out_bf16;
  int out_wide;     // out lies at a multiple of 32 bytes
  float* part_o;    // [2 CTAs][TILES][D / 4][128 rows][4], normalised
  float* part_lse;  // [2 CTAs][TILES * 128], log2
  TreeStart* start; // [CTAs]
  int num_seqs, total_q, max_q_len, q_heads, kv_heads, num_blocks, max_blocks_per_seq;
  int lanes;  // parts of the grid that take the KV heads side by side
  float scale_log2;
};

// A sequence's share of the work: row groups and key tiles (0 groups: none).
struct TreeSeq {
  int qs, n, ctx, groups, tiles;
  bool bad;
  __device__ __forceinline__ int total(int heads) const { return groups * tiles * heads; }
  // With kTrSlack places before each item for what its start costs: places, and
  // the key tiles among the first x of them.
  __device__ __forceinline__ int places(int heads) const {
    return groups * (tiles + kTrSlack) * heads;
  }
  __device__ __forceinline__ int tiles_in(int x, int heads) const {
    x = min(max(x, 0), places(heads));
    const int item = x / (tiles + kTrSlack);
    return item * tiles + max(x - item * (tiles + kTrSlack) - kTrSlack, 0);
  }
};

template <int G, int TILES>
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int s) {
  TreeSeq r;
  r.qs = __ldg(p.q_start + s);
  const int qe = __ldg(p.q_start + s + 1);
  r.ctx = __ldg(p.context_lens + s);
  r.n = qe - r.qs;
  r.bad = r.qs < 0 || r.n < 0 || qe > p.total_q || r.n > p.max_q_len || r.n > r.ctx ||
          r.ctx > p.max_blocks_per_seq * 16;
  constexpr int kTokens = TILES * kTrRows / G;
  r.groups = r.bad ? 0 : (r.n + kTokens - 1) / kTokens;
  r.tiles = r.bad ? 0 : (r.ctx + kTrKeys - 1) / kTrKeys;
  return r;
}

// A piece of an item in a CTA's range, as the softmax and P V warps take it
// (tiles 0: no more).
struct TreePiece {
  int qs, n, ctx, seq, kvh, node0, first, tiles;  // tiles < 0: the whole item
};

// The pieces of items in one CTA's range, in order.
template <int G, int TILES>
struct TreeWalk {
  const TreeParams& p;
  int s;
  int off;         // tiles of sequence s before the next piece
  int lane, heads; // part of the grid and its KV heads: lane, lane + lanes, ...
  int left;        // tiles of the range after the current piece
  TreeSeq seq;
  int item, first, tiles;  // current piece
  __device__ __forceinline__ TreeWalk(const TreeParams& pp, const TreeSeq& q0, int s0,
                                      int off0, int count, int lane0, int heads0)
      : p(pp), s(s0), off(off0), lane(lane0), heads(heads0), left(count), seq(q0) {}
  __device__ __forceinline__ bool next() {
    if (left <= 0) return false;
    while (off >= seq.total(heads)) {
      if (++s >= p.num_seqs) return false;
      off = 0;
      seq = tree_seq<G, TILES>(p, s);
    }
    item = off / seq.tiles;
    first = off - item * seq.tiles;
    tiles = min(seq.tiles - first, left);
    off += tiles;
    left -= tiles;
    return true;
  }
  __device__ __forceinline__ int kv_head() const {
    return lane + item / seq.groups * p.lanes;
  }
  __device__ __forceinline__ int group() const { return item % seq.groups; }
  __device__ __forceinline__ bool whole() const { return first == 0 && tiles == seq.tiles; }
};

// Bounded wait that also gives up as soon as another role has aborted.
__device__ __forceinline__ bool tr_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  for (uint32_t i = 0; i < kWaitPollLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 255u && *abort_flag) return false;
  }
  return false;
}

__device__ __forceinline__ void tr_abort(volatile int* abort_flag) {
  *abort_flag = 1;
  atomicOr(&g_tree_error, kErrWaitTimeout);
}

// 32 of a row's key bits: key0 + i - base is node i's distance into the tree.
__device__ __forceinline__ uint32_t key_bits(unsigned long long mask, int off) {
  if (off >= 64 || off <= -32) return off < 0 ? 0xffffffffu : 0u;
  if (off >= 0) return uint32_t(mask >> off);
  return ((1u << -off) - 1u) | uint32_t(mask << -off);
}

// 32 bytes to a multiple of 16, in one piece where it is one of 32.
__device__ __forceinline__ void store_sector(void* to, const uint32_t (&y)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(y[0]),
                 "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                 : "memory");
  } else {
    static_cast<uint4*>(to)[0] = make_uint4(y[0], y[1], y[2], y[3]);
    static_cast<uint4*>(to)[1] = make_uint4(y[4], y[5], y[6], y[7]);
  }
}

__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_u4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w) : "memory");
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

// The bits 15 and 31 of the halves of a bf16 pair that are NaN or infinite.
__device__ __forceinline__ uint32_t nonfinite_bf16x2(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ uint32_t keep_finite(uint32_t w) {
  return w & ~((nonfinite_bf16x2(w) >> 15) * 0xffffu);
}

// 32 columns of this thread's tensor-memory lane; the registers hold them after
// the next tmem_wait_ld, which may be many instructions later.
__device__ __forceinline__ void tmem_ld32u(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}

// 32 scores to weights 2^(x sc - m) as bf16 hi + lo pairs, in place: of each
// 16 scores hi in the first 8 registers, lo in the others.  Adds the weights
// to ls.
__device__ __forceinline__ void tree_weigh(uint32_t (&v)[32], uint64_t sc2, uint64_t nm2,
                                           uint64_t (&ls)[2]) {
#pragma unroll
  for (int b = 0; b < 32; b += 16) {
    uint32_t lo[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      float x0, x1, e0, e1, r0, r1;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(v[b + 2 * u]), __uint_as_float(v[b + 2 * u + 1])),
                       sc2, nm2), x0, x1);
      const uint64_t e = f2_pack(ex2(x0), ex2(x1));
      ls[u & 1] = f2_add(ls[u & 1], e);
      f2_unpack(e, e0, e1);
      const uint32_t h = pack_bf16x2(e0, e1);
      f2_unpack(f2_sub(e, f2_pack(bf16_lo_to_f32(h), bf16_hi_to_f32(h))), r0, r1);
      v[b + u] = h;
      lo[u] = pack_bf16x2(r0, r1);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) v[b + 8 + u] = lo[u];
  }
}

template <int D, int G, int TILES>
__global__ void __launch_bounds__(kTrThreads, 1)
paged_tree_kernel(const __grid_constant__ CUtensorMap tmap_q,
                  const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v, const TreeParams p) {
  using T = TreeSmem<D, TILES>;
  constexpr int TPT = kTrRows / G;  // tree nodes per row tile
  constexpr int kParts = T::kParts;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + T::kBarOff;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + T::kMiscOff + 4);
  unsigned long long* nonfinite = reinterpret_cast<unsigned long long*>(smem + T::kMiscOff + 16);
  int* scan = reinterpret_cast<int*>(smem + T::kMiscOff + 32);
  struct Begin {
    TreeSeq seq;
    int s, off, count;
  };
  static_assert(sizeof(Begin) <= 48, "start of the range");
  volatile TreePiece* pieces = reinterpret_cast<volatile TreePiece*>(smem + T::kPieceOff);
  Begin* begin = reinterpret_cast<Begin*>(smem + T::kMiscOff + 80);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- set-up that reads no input, beside the previous kernel's end
  griddep_launch_dependents();  // the merge waits for this grid before it reads
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), kTrTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == kTrKWarp * 32) {
    mbar_init(bars + 8 * kTrQFull, 1);
    mbar_init(bars + 8 * kTrQEmpty, 1);
#pragma unroll 1
    for (int s = 0; s < kTrMaxStages; ++s) {
      mbar_init(bars + 8 * (kTrKFull + s), 1);
      mbar_init(bars + 8 * (kTrKEmpty + s), 1);
      mbar_init(bars + 8 * (kTrVFull + s), 1);
      mbar_init(bars + 8 * (kTrVEmpty + s), 1);
    }
    for (int h = 0; h < 6; ++h) {
      mbar_init(bars + 8 * (kTrSFull + h), 1);
      mbar_init(bars + 8 * (kTrPFull + h), 4);
      mbar_init(bars + 8 * (kTrDone + h), 1);
    }
    mbar_init(bars + 8 * kTrXch, 8);
    mbar_init(bars + 8 * kTrEpi, 8);
    mbar_init(bars + 8 * kTrDrain, 2);
    for (int s = 0; s < kTrPieces; ++s) mbar_init(bars + 8 * (kTrPiece0 + s), 1);
    fence_barrier_init();
    *abort_flag = 0;
    nonfinite[0] = nonfinite[1] = 0;
    begin->count = 0;
  }
  if (threadIdx.x == kTrVWarp * 32) tma_prefetch_desc(&tmap_v);
  if (threadIdx.x == kTrSWarp * 32) {
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_q);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // inputs may have been written by the previous kernel in the stream

  // ---- this CTA's range of the key tiles of all items
  // The grid's `lanes` equal parts take a share of the KV heads each.  Where there
  // is work for some CTAs only, they then lie all over the GPU (us, against one
  // part: 1 x 500 11.8 / 12.4, 1 x 2000 15.4 / 16.8, 4 x 1000 16.7 / 17.4, 16 x 4096
  // 50.7 / 51.8, 2 x 131072 with heads of 64 107 / 137; 64 x 8192 the same).  CTAs that
  // the division leaves over have no work.
  const int ctas = gridDim.x / p.lanes, heads = p.kv_heads / p.lanes;
  const int part = blockIdx.x / ctas;
  const int c = part < p.lanes ? blockIdx.x - part * ctas : ctas;
  TreeSeq q{};               // the sequence it starts in,
  int s0 = -1, off0 = 0;     // its number, and the tiles of it before the range
  int count = 0;
  auto warp_scan = [&](int x) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += up;
    }
    return x;
  };
  // The items' places laid end to end, CTA c starting at floor(c all / active).
  // With few the last CTAs have none.  A CTA whose places hold no tile has no
  // work; a cut item's pieces lie in consecutive CTAs all the same.
  auto even_share = [&](int all, int& lo, int& n) {
    constexpr int kLeast = kTrMinTiles + kTrSlack;
    const int active = min(ctas, (all + kLeast - 1) / kLeast);
    const int each = active > 0 ? all / active : 0, rest = all - each * active;
    lo = c < active ? c * each + c * rest / active : all;
    n = c < active ? (c + 1) * each + (c + 1) * rest / active - lo : 0;
  };
  if (p.num_seqs <= 32) {
    // every warp for itself, lane = sequence: no barrier before the first load
    if (lane < p.num_seqs) q = tree_seq<G, TILES>(p, lane);
    if (q.bad && blockIdx.x == 0 && warp == 0) atomicOr(&g_tree_error, kErrBadQueryRange);
    const int items = q.groups * heads;
    const int tiles = __reduce_add_sync(0xffffffffu, q.total(heads));
    // With no more items than CTAs each item is cut into equal pieces of at most
    // kTrSlack tiles above the even share, one piece a CTA, if there are CTAs
    // enough.
    const int longest = max(kTrMinTiles, tiles / ctas + kTrSlack);
    const int cuts =
        items ? max(1, min((q.tiles + longest - 1) / longest, q.tiles / kTrMinTiles)) : 0;
    const bool alone = __reduce_add_sync(0xffffffffu, items * cuts) <= ctas;
    const int width = alone ? items * cuts : q.places(heads);
    const int end = warp_scan(width);
    int lo = c, n = 0;
    if (!alone) even_share(__shfl_sync(0xffffffffu, end, 31), lo, n);
    const int at = lo - (end - width);
    if (!alone)
      count = __reduce_add_sync(0xffffffffu, q.tiles_in(at + n, heads) -
                                                 q.tiles_in(at, heads));
    const unsigned here = __ballot_sync(0xffffffffu, at >= 0 && at < width);
    if (here) {
      const int src = __ffs(here) - 1;
      if (alone && lane == src) {
        const int item = at / cuts, j = at - item * cuts, first = j * q.tiles / cuts;
        off0 = item * q.tiles + first;
        count = (j + 1) * q.tiles / cuts - first;
      } else {
        off0 = q.tiles_in(at, heads);
      }
      s0 = src;
      off0 = __shfl_sync(0xffffffffu, off0, src);
      count = __shfl_sync(0xffffffffu, count, src);  // the same in all lanes if not alone
      q.qs = __shfl_sync(0xffffffffu, q.qs, src);
      q.n = __shfl_sync(0xffffffffu, q.n, src);
      q.ctx = __shfl_sync(0xffffffffu, q.ctx, src);
      q.groups = __shfl_sync(0xffffffffu, q.groups, src);
      q.tiles = __shfl_sync(0xffffffffu, q.tiles, src);
    } else {
      count = 0;
    }
  } else {
    const int per_thread = (p.num_seqs + kTrThreads - 1) / kTrThreads;
    const int s_lo = min(int(threadIdx.x) * per_thread, p.num_seqs);
    const int s_hi = min(s_lo + per_thread, p.num_seqs);
    int mine = 0;
    for (int s = s_lo; s < s_hi; ++s) {
      q = tree_seq<G, TILES>(p, s);
      if (q.bad && blockIdx.x == 0) atomicOr(&g_tree_error, kErrBadQueryRange);
      mine += q.places(heads);
    }
    int incl = warp_scan(mine), all = 0, lo, n;
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTrThreads / 32; ++w) {
      if (w == warp) incl += all;
      all += scan[w];
    }
    even_share(all, lo, n);
    if (lo < incl && lo + n > incl - mine) {  // some of the range is this thread's
      int at = lo - (incl - mine);
      for (int s = s_lo; s < s_hi; ++s) {
        if (per_thread > 1) q = tree_seq<G, TILES>(p, s);
        const int tiles = q.tiles_in(at + n, heads) - q.tiles_in(at, heads);
        if (tiles > 0) atomicAdd(&begin->count, tiles);
        if (at >= 0 && at < q.places(heads)) {  // it starts here
          begin->seq = q;
          begin->s = s;
          begin->off = q.tiles_in(at, heads);
        }
        at -= q.places(heads);
      }
    }
    __syncthreads();
    count = begin->count;
    if (count > 0) {
      q = begin->seq;
      s0 = begin->s;
      off0 = begin->off;
    }
  }
  if (threadIdx.x == 0) {
    TreeStart at{-1, 0, 0, 0, 0, 0, {0, 0}};
    if (count > 0) {
      const int item = off0 / q.tiles, kvh = part + item / q.groups * p.lanes;
      at = TreeStart{s0, kvh * q.groups + item % q.groups, off0 - item * q.tiles, q.qs, q.n,
                     q.groups, {0, 0}};
    }
    p.start[blockIdx.x] = at;
  }
  if (count > 0) {
  TreeWalk<G, TILES> walk(p, q, s0, off0, count, part, heads);

  // The launch gives every warp 168 registers; the four loading and issuing
  // warps hand some of theirs to the softmax warps.  8 x 192 + 4 x 120 <= 12 x 168
  // (checked at the launch).
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTrRegsIssue));
  if (warp == kTrKWarp || warp == kTrVWarp) {
    // ================= K and V rings =================
    const bool is_v = warp == kTrVWarp;
    const int stages = is_v ? T::kVStages : T::kKStages;
    const uint32_t ring = sbase + (is_v ? T::kVOff : T::kKOff);
    const uint32_t full = bars + 8 * (is_v ? kTrVFull : kTrKFull);
    const uint32_t empty = bars + 8 * (is_v ? kTrVEmpty : kTrKEmpty);
    const CUtensorMap* map = is_v ? &tmap_v : &tmap_k;
    constexpr int kLoads = 8 * (D / 64);  // pages x column halves
    int i = 0;
    bool ok = true;
    while (ok && walk.next()) {
      const int kvh = walk.kv_head();
      const int32_t* table = p.block_tables + size_t(walk.s) * p.max_blocks_per_seq;
      const int nblk = (walk.seq.ctx + 15) / 16;
      for (int j = 0; j < walk.tiles; ++j, ++i) {
        const int st = i % stages;
        const int blk0 = (walk.first + j) * 8, blk = blk0 + lane / (D / 64);
        int id = -1;  // pages past the context: the box is out of bounds and reads zeros
        if (lane < kLoads && blk < nblk) {
          id = __ldg(table + blk);
          if (id < 0 || id >= p.num_blocks) {
            atomicOr(&g_tree_error, kErrBadBlockId);
            id = -1;
          }
        }
        // The table's next entries come into L2 four tiles before they are
        // read: without it a read of a new line took 4000-5700 cycles behind
        // the queued pages, every fourth tile.
        if (lane == 0 && !is_v && blk0 % 32 == 0 && blk0 + 32 < nblk)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(table + blk0 + 32));
        if (i >= stages) {
          ok = __all_sync(0xffffffffu, tr_wait(empty + 8 * st, (i / stages - 1) & 1, abort_flag));
          if (!ok) break;
        }
        if (lane == 0) mbar_arrive_expect_tx(full + 8 * st, T::kTileBytes);
        __syncwarp();
        if (lane < kLoads)
          tma_load_4d(ring + st * T::kTileBytes + (lane % (D / 64)) * T::kHalf +
                          (lane / (D / 64)) * 2048,
                      map, full + 8 * st, (lane % (D / 64)) * 64, kvh, 0, id);
      }
    }
    if (!ok) {
      // no copy may land after the CTA exits: wait (bounded) for the last one
      // of each slot
      if (lane == 0) {
        tr_abort(abort_flag);
        for (int k = max(0, i - stages); k < i; ++k)
          (void)mbar_wait_bounded(full + 8 * (k % stages), (k / stages) & 1);
      }
    } else if (lane == 0) {
      // the last release of each slot has arrived before the CTA exits (or,
      // after an abort elsewhere, the copies have)
      for (int k = max(0, i - stages); k < i; ++k) {
        if (!tr_wait(empty + 8 * (k % stages), (k / stages) & 1, abort_flag))
          (void)mbar_wait_bounded(full + 8 * (k % stages), (k / stages) & 1);
      }
    }
    __syncwarp();
  } else if (warp == kTrSWarp) {
    // ================= Q, and the products S = Q K^T =================
    // S and P V are issued by two warps, so that one's waits and the other's
    // MMAs overlap.  Each runs as a whole warp and elects a lane for the MMAs:
    // descriptors are then values of the warp.  From a branch on the lane number
    // an MMA took 75-90 cycles to issue, more than it runs for with heads of 64
    // (2 x 131072, 27 nodes: 128 us against 110).
    constexpr uint32_t kIdesc = idesc_bf16_f32(128, kTrKeys / kParts, 0, 0);
    auto wait = [&](int bar, uint32_t parity) {
      return bool(__all_sync(0xffffffffu, tr_wait(bars + 8 * bar, parity, abort_flag)));
    };
    int i = 0, k = 0;
    bool ok = true;
    // The pieces are worked out here, ahead of those who need them.  Slot k
    // is free: the last S product needed a P V of piece k - 4 or later, whose
    // first one needed everybody to be through with piece k - 5.
    auto publish = [&](bool some) {
      volatile TreePiece* t = pieces + k % kTrPieces;
      if (some && lane == 0) {
        t->qs = walk.seq.qs;
        t->n = walk.seq.n;
        t->ctx = walk.seq.ctx;
        t->seq = walk.s;
        t->kvh = walk.kv_head();
        t->node0 = walk.group() * TILES * TPT;
        t->first = walk.first;
      }
      if (lane == 0) {
        t->tiles = some ? (walk.whole() ? -walk.tiles : walk.tiles) : 0;
        mbar_arrive(bars + 8 * (kTrPiece0 + k % kTrPieces));
      }
      __syncwarp();
    };
    for (; ok; ++k) {
      const bool some = walk.next();
      publish(some);
      if (!some) break;
      ok = k == 0 || wait(kTrQEmpty, (k - 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bars + 8 * kTrQFull, T::kQBytes);
        const int tok = walk.seq.qs + walk.group() * TILES * TPT;
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(sbase + t * T::kTileBytes + h * T::kHalf, &tmap_q, bars + 8 * kTrQFull,
                        h * 64, walk.kv_head() * G, tok + t * TPT);
      }
      __syncwarp();
      ok = wait(kTrQFull, k & 1);
#pragma unroll 1
      for (int j = 0; ok && j < walk.tiles; ++j, ++i) {
        ok = wait(kTrKFull + i % T::kKStages, (i / T::kKStages) & 1);
        // a part's columns are free once the products that read its P are done
#pragma unroll 1
        for (int th = 0; ok && th < kParts * TILES; ++th) {
          const int t = th / kParts, h = th % kParts, job = i * TILES + t;
          const int b = job % T::kBufs, before = job / T::kBufs - 1;
          ok = before < 0 || wait(kTrDone + 3 * h + b, before & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t q_smem = sbase + t * T::kTileBytes;
          const uint32_t k_smem =
              sbase + T::kKOff + (i % T::kKStages) * T::kTileBytes + h * 64 * 128;
          if (elect_lane()) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              const uint32_t off = (c >> 2) * T::kHalf + (c & 3) * 32;
              umma_bf16(tmem + T::buf_col(b) + h * 64, smem_desc_sw128(q_smem + off, 16, 1024),
                        smem_desc_sw128(k_smem + off, 16, 1024), kIdesc, c > 0);
            }
            umma_commit(bars + 8 * (kTrSFull + 3 * h + b));
          }
        }
        if (elect_lane()) {
          umma_commit(bars + 8 * (kTrKEmpty + i % T::kKStages));
          if (j + 1 == walk.tiles) umma_commit(bars + 8 * kTrQEmpty);
        }
      }
    }
    if (!ok && lane == 0) tr_abort(abort_flag);
    // every MMA issued has completed, and Q has landed, before the CTA exits
    if (elect_lane()) umma_commit(bars + 8 * kTrDrain);
    (void)mbar_wait_bounded(bars + 8 * kTrDrain, 0);
    if (!ok && k > 0) (void)mbar_wait_bounded(bars + 8 * kTrQFull, (k - 1) & 1);
    __syncwarp();
  } else {
    // ================= the products O += P V =================
    constexpr uint32_t kIdesc = idesc_bf16_f32(128, D, 0, 1);
    auto wait = [&](int bar, uint32_t parity) {
      return bool(__all_sync(0xffffffffu, tr_wait(bars + 8 * bar, parity, abort_flag)));
    };
    int i = 0;
    bool ok = true;
    int k = 0;
    for (; ok; ++k) {
      ok = wait(kTrPiece0 + k % kTrPieces, (k / kTrPieces) & 1);
      const int tiles = ok ? abs(pieces[k % kTrPieces].tiles) : 0;
      if (tiles == 0) break;
      if (k > 0) ok = wait(kTrEpi, (k - 1) & 1);  // the accumulators have been read
#pragma unroll 1
      for (int j = 0; ok && j < tiles; ++j, ++i) {
        const bool fresh = j < (TILES == 1 ? 2 : 1);  // the accumulator's first tile of the piece
        ok = wait(kTrVFull + i % T::kVStages, (i / T::kVStages) & 1);
        const uint32_t v_smem = sbase + T::kVOff + (i % T::kVStages) * T::kTileBytes;
#pragma unroll 1
        for (int th = 0; ok && th < kParts * TILES; ++th) {
          const int t = th / kParts, h = th % kParts, job = i * TILES + t;
          const int b = job % T::kBufs;
          ok = wait(kTrPFull + 3 * h + b, (job / T::kBufs) & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_lane()) {
#pragma unroll
            for (int c = 0; c < kTrKeys / 16 / kParts; ++c) {
              const uint64_t vdesc = smem_desc_sw128(v_smem + (4 * h + c) * 2048, T::kHalf, 1024);
              // hi, and lo 8 columns on
              const uint32_t a_hi = tmem + T::buf_col(b) + 64 * h + 16 * c;
              umma_bf16_ts(tmem + T::out_col(job & 1), a_hi, vdesc, kIdesc,
                           (!fresh || h > 0 || c > 0) ? 1u : 0u);
              umma_bf16_ts(tmem + T::out_col(job & 1), a_hi + 8, vdesc, kIdesc, 1u);
            }
            umma_commit(bars + 8 * (kTrDone + 3 * h + b));
          }
        }
        if (!ok) break;
        if (elect_lane()) umma_commit(bars + 8 * (kTrVEmpty + i % T::kVStages));
      }
    }
    if (!ok && lane == 0) tr_abort(abort_flag);
    if (elect_lane()) umma_commit(bars + 8 * kTrDrain);
    (void)mbar_wait_bounded(bars + 8 * kTrDrain, 0);
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTrRegsSoftmax));
    // ================= softmax, correction, epilogue =================
    const int w = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the tile = tensor-memory lane
    const uint32_t lane_base = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t o_col = T::out_col(w);
    float2* xch = reinterpret_cast<float2*>(smem + T::kXchOff);
    const bool neg = p.scale_log2 < 0.f;  // uniform
    const float mag = fabsf(p.scale_log2);
    int i = 0;  // stream tile the current piece begins at
    bool ok = true;
    for (int k = 0;; ++k) {
      ok = __all_sync(0xffffffffu, tr_wait(bars + 8 * (kTrPiece0 + k % kTrPieces),
                                           (k / kTrPieces) & 1, abort_flag));
      if (!ok) break;
      const volatile TreePiece* piece = pieces + k % kTrPieces;
      const int n = piece->n, ctx = piece->ctx, first = piece->first, tiles = abs(piece->tiles);
      if (tiles == 0) break;
      const int node0 = piece->node0 + (TILES == 2 ? w : 0) * TPT;  // of the tile
      const int node = node0 + r / G;
      const bool valid = node < n;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      const int base = ctx - n;  // committed keys
      // as loaded: cut to the nodes where it is used, so that nobody waits for it here
      const unsigned long long raw_mask =
          __ldg(p.tree_mask + piece->qs + (valid ? node : n - 1));
      const unsigned long long nodes =
          !valid ? 0ull : n < 64 ? (1ull << n) - 1ull : ~0ull;
      float m = -INFINITY, l = 0.f;
      int seen = 0;  // tiles of the piece this warpgroup has taken
      for (int j = 0; j < tiles; ++j) {
        const int it = i + j;
        if (TILES == 1 && (it & 1) != w) continue;
        const int job = TILES == 1 ? it : 2 * it + w, b = job % T::kBufs, ph = job / T::kBufs;
        const uint32_t s_col = T::buf_col(b);
        const int key0 = (first + j) * kTrKeys;
        const bool masked = key0 + kTrKeys > base;
        if (masked && (TILES == 1 || w == 0)) {
          // thread r looks at key row r of V; the chunk order differs from
          // row to row, so that a warp's reads spread over the banks.
          // S comes first: a wait on a parity says something only once the phase before is
          // over, here the copy of tile it - kVStages into the same slot.  S of this job
          // was issued after the products of job - kBufs, and those, in their order, after
          // that tile's.
          ok = __all_sync(0xffffffffu,
                          tr_wait(bars + 8 * (kTrSFull + b), ph & 1, abort_flag));
          if (!ok) break;
          ok = __all_sync(0xffffffffu, tr_wait(bars + 8 * (kTrVFull + it % T::kVStages),
                                               (it / T::kVStages) & 1, abort_flag));
          if (!ok) break;
          const int key = key0 + r;
          if (key >= base) {
            const uint32_t row = sbase + T::kVOff + (it % T::kVStages) * T::kTileBytes + r * 128;
            uint32_t any = 0;
#pragma unroll 1
            for (int h = 0; h < D / 64; ++h)
#pragma unroll 4
              for (int c = 0; c < 8; ++c) {
                const uint32_t at = row + h * T::kHalf + (((c + r) & 7) << 4);
                const uint4 v = ld_shared_u4(at);
                const uint32_t bad = nonfinite_bf16x2(v.x) | nonfinite_bf16x2(v.y) |
                                     nonfinite_bf16x2(v.z) | nonfinite_bf16x2(v.w);
                if (bad) {
                  st_shared_u4(at, make_uint4(keep_finite(v.x), keep_finite(v.y),
                                              keep_finite(v.z), keep_finite(v.w)));
                  any = 1;
                }
              }
            if (any) {
              if (key < ctx) atomicOr(nonfinite + (k & 1), 1ull << (key - base));
              fence_proxy_async_smem();
            }
          }
        }
#pragma unroll 1
        for (int c = 0; c < kTrKeys; c += 64) {  // the halves of the tile
          const int h = c >> 6;
          if (kParts == 2 || h == 0) {
            ok = __all_sync(0xffffffffu,
                            tr_wait(bars + 8 * (kTrSFull + 3 * h + b), ph & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
          }
          if (warp_valid) {
            uint32_t va[32], vb[32];
            if (masked) {
              // hidden keys' scores become what weighs nothing: -inf after scaling
              const uint32_t hide = __float_as_uint(neg ? INFINITY : -INFINITY);
#pragma unroll 1
              for (int cc = c; cc < c + 64; cc += 32) {
                const uint32_t bits = key_bits(raw_mask & nodes, key0 + cc - base);
                tmem_ld32u(lane_base + s_col + cc, va);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 32; ++u) va[u] = (bits >> u) & 1u ? va[u] : hide;
                tmem_st32u(lane_base + s_col + cc, va);
              }
              tmem_wait_st();
            }
            // The running max m is a reference only: any value near the scores'
            // serves.  So the keys are weighed against the m it has, without
            // looking for their max, and that stands while each row's sum is at
            // most kTrMaxSum.  Where no key has been seen yet, or a sum is larger,
            // the max is taken first, and m moves when it is more than 8 behind (a
            // factor 256).
            const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
            bool raise = !__all_sync(0xffffffffu, m != -INFINITY);
#pragma unroll 1
            for (;;) {
              tmem_ld32u(lane_base + s_col + c, va);
              tmem_ld32u(lane_base + s_col + c + 32, vb);
              tmem_wait_ld();
              if (raise) {
                float ex[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                const uint32_t flip = neg ? 0x80000000u : 0u;
#pragma unroll
                for (int u = 0; u < 32; ++u)
                  ex[u & 3] = max3f(ex[u & 3], __uint_as_float(va[u] ^ flip),
                                    __uint_as_float(vb[u] ^ flip));
                const float top = fmaxf(fmaxf(ex[0], ex[1]), fmaxf(ex[2], ex[3]));
                const float mx = top == -INFINITY ? -INFINITY : top * mag;
                const bool move = mx > m + kTrRescale || (m == -INFINITY && mx > m);
                if (__any_sync(0xffffffffu, move)) {
                  const float alpha = move ? ex2(m - mx) : 1.f;  // 0 when m is -inf
                  if (seen > 0 || (kParts == 2 && h > 0)) {
                    // the accumulator's last products must be done before it is scaled
                    const bool own = kParts == 2 && h > 0;  // of the tile's first half
                    const int of = own ? job : job - 2;
                    ok = __all_sync(0xffffffffu,
                                    tr_wait(bars + 8 * (kTrDone + (own ? 0 : 3 * (kParts - 1)) +
                                                        of % T::kBufs),
                                            (of / T::kBufs) & 1, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll 1
                    for (int cc = 0; cc < D; cc += 32) {
                      tmem_ld32u(lane_base + o_col + cc, va);
                      tmem_wait_ld();
#pragma unroll
                      for (int u = 0; u < 32; u += 2) {
                        float y0, y1;
                        f2_unpack(f2_mul(f2_pack(__uint_as_float(va[u]),
                                                 __uint_as_float(va[u + 1])), a2), y0, y1);
                        va[u] = __float_as_uint(y0), va[u + 1] = __float_as_uint(y1);
                      }
                      tmem_st32u(lane_base + o_col + cc, va);
                    }
                  }
                  if (kParts == 1 && h > 0) {  // so is the P of the first half, still unused
                    tmem_wait_st();
#pragma unroll 1
                    for (int cc = 0; cc < 64; cc += 32) {
                      tmem_ld32u(lane_base + s_col + cc, va);
                      tmem_wait_ld();
#pragma unroll
                      for (int u = 0; u < 32; u += u % 8 == 7 ? 9 : 1) {
                        const uint32_t h = va[u], lw = va[u + 8];
                        const float e0 = (bf16_lo_to_f32(h) + bf16_lo_to_f32(lw)) * alpha;
                        const float e1 = (bf16_hi_to_f32(h) + bf16_hi_to_f32(lw)) * alpha;
                        va[u] = pack_bf16x2(e0, e1);
                        va[u + 8] =
                            pack_bf16x2(e0 - bf16_lo_to_f32(va[u]), e1 - bf16_hi_to_f32(va[u]));
                      }
                      tmem_st32u(lane_base + s_col + cc, va);
                    }
                  }
                  tmem_ld32u(lane_base + s_col + c, va);
                  tmem_wait_ld();
                  l *= alpha;
                  if (move) m = mx;
                }
              }
              // P = 2^(x - m) as bf16 hi + lo in the scores' place: of each 16 keys
              // hi in the first 8 columns, lo in the others, two keys a column
              const float mref = m == -INFINITY ? 0.f : m;  // nothing seen yet: all P are 0
              const uint64_t nm2 = f2_pack(-mref, -mref);
              uint64_t ls[2] = {0ull, 0ull};
              tree_weigh(va, sc2, nm2, ls);
              tree_weigh(vb, sc2, nm2, ls);
              float a0, a1, b0, b1;
              f2_unpack(ls[0], a0, a1);
              f2_unpack(ls[1], b0, b1);
              const float sum = (a0 + a1) + (b0 + b1);
              if (raise || __all_sync(0xffffffffu, sum <= kTrMaxSum)) {
                l += sum;
                break;
              }
              raise = true;  // NaN, too; the scores are still there
            }
            if (!ok) break;
            tmem_st32u(lane_base + s_col + c, va);
            tmem_st32u(lane_base + s_col + c + 32, vb);
          }
          if (kParts == 2 || h > 0) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + 8 * (kTrPFull + 3 * (kParts - 1 ? h : 0) + b));
          }
        }
        if (!ok) break;
        ++seen;
      }
      if (!ok) break;

      // ---- end of the piece: both warpgroups meet
      if (k > 0) {  // the exchange of the piece before has been read
        ok = __all_sync(0xffffffffu, tr_wait(bars + 8 * kTrEpi, (k - 1) & 1, abort_flag));
        if (!ok) break;
      }
      if (warp == 0 && lane == 0) nonfinite[(k + 1) & 1] = 0;
      xch[w * kTrRows + r] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * kTrXch);
      ok = __all_sync(0xffffffffu, tr_wait(bars + 8 * kTrXch, k & 1, abort_flag));
      if (!ok) break;
      // both accumulators' last products of the piece are done: each may be
      // read, and nobody reads the last V tile any more
      const int begin_tile = i;
      i += tiles;
#pragma unroll 1
      for (int a = 0; a < 2; ++a) {
        const int lt = TILES == 2 || ((i - 1) & 1) == a ? i - 1 : i - 2;  // its last tile
        if (lt < begin_tile) continue;
        const int job = TILES == 1 ? lt : 2 * lt + a;
        ok = __all_sync(0xffffffffu,
                        tr_wait(bars + 8 * (kTrDone + 3 * (kParts - 1) + job % T::kBufs),
                                (job / T::kBufs) & 1, abort_flag));
        if (!ok) break;
      }
      if (!ok) break;
      float fa = 0.f, fb = 0.f, lse = -INFINITY;  // factors of O_w and of the other O
      if constexpr (TILES == 1) {
        const float2 other = xch[(1 - w) * kTrRows + r];
        const float big = fmaxf(m, other.x);
        const float ref = big == -INFINITY ? 0.f : big;
        const float wa = ex2(m - ref), wb = ex2(other.x - ref);
        const float tot = l * wa + other.y * wb;
        if (l != 0.f) fa = wa / tot;  // NaN scores included
        if (other.y != 0.f) fb = wb / tot;
        if (tot != 0.f) lse = ref + __log2f(tot);
      } else if (l != 0.f) {
        fa = 1.f / l;
        lse = (m == -INFINITY ? 0.f : m) + __log2f(l);
      }
      tc_fence_after();

      // TILES 1: this warpgroup's half of the columns of both accumulators.  They
      // are read in groups of up to 64, as many as the registers hold; with the
      // last group read, before it is stored, the accumulators are free for the
      // next piece's products.
      constexpr int kAll = TILES == 1 ? D / 2 : D, kCols = kAll < 64 ? kAll : 64;
      const int qs = piece->qs, seq = piece->seq, kvh = piece->kvh;
      const bool whole = piece->tiles < 0;
      const unsigned long long hit = raw_mask & nodes & nonfinite[k & 1];
      const bool use_a = __any_sync(0xffffffffu, fa != 0.f);
      const bool use_b = TILES == 1 && __any_sync(0xffffffffu, fb != 0.f);
#pragma unroll 1
      for (int g = 0; g < kAll; g += kCols) {
        const int col0 = (TILES == 1 ? w * kAll : 0) + g;
        uint32_t o[kCols / 32][32];
        if (warp_valid) {
          // an accumulator that no tile of the piece went to holds anything
          if (use_a) {
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c)
              tmem_ld32u(lane_base + o_col + col0 + 32 * c, o[c]);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c)
#pragma unroll
              for (int u = 0; u < 32; ++u) o[c][u] = 0;
          }
          const uint64_t a2 = f2_pack(fa, fa), b2 = f2_pack(fb, fb);
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c)
#pragma unroll
            for (int u = 0; u < 32; u += 2) {
              float y0, y1;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(o[c][u]), __uint_as_float(o[c][u + 1])), a2),
                        y0, y1);
              o[c][u] = __float_as_uint(y0), o[c][u + 1] = __float_as_uint(y1);
            }
          if (use_b) {
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c) {
              uint32_t x[32];
              tmem_ld32u(lane_base + T::out_col(1 - w) + col0 + 32 * c, x);
              tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 32; u += 2) {
                float y0, y1;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(x[u]), __uint_as_float(x[u + 1])), b2,
                                 f2_pack(__uint_as_float(o[c][u]), __uint_as_float(o[c][u + 1]))),
                          y0, y1);
                o[c][u] = __float_as_uint(y0), o[c][u + 1] = __float_as_uint(y1);
              }
            }
          }
        }
        if (g + kCols == kAll) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + 8 * kTrEpi);
        }
        if (valid) {
          if (!whole) {
            // A cut item's rows go to the workspace in quads of columns, 512 contiguous
            // bytes a store.  Slot 2c: the piece the CTA's range starts with, 2c + 1: the
            // one it ends with.
            const size_t tile = (size_t(blockIdx.x) * 2 + (k == 0 ? 0 : 1)) * TILES +
                                (TILES == 2 ? w : 0);
            uint4* to =
                reinterpret_cast<uint4*>(p.part_o) + (tile * (D / 4) + col0 / 4) * kTrRows + r;
#pragma unroll
            for (int u = 0; u < kCols; u += 4)
              to[u / 4 * kTrRows] = make_uint4(o[u / 32][u % 32], o[u / 32][u % 32 + 1],
                                               o[u / 32][u % 32 + 2], o[u / 32][u % 32 + 3]);
            if (col0 == 0) p.part_lse[tile * kTrRows + r] = lse;
          }
          // A whole item's rows go out as sectors of 32 bytes.
          const size_t out0 =
              ((size_t(qs) + node) * p.q_heads + size_t(kvh) * G + r % G) * D + col0;
          if (whole && p.out_bf16) {
            __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + out0;
#pragma unroll
            for (int u = 0; u < kCols; u += 16) {
              uint32_t y[8];
#pragma unroll
              for (int v = 0; v < 8; ++v)
                y[v] = pack_bf16x2(__uint_as_float(o[u / 32][u % 32 + 2 * v]),
                                   __uint_as_float(o[u / 32][u % 32 + 2 * v + 1]));
              store_sector(to + u, y, p.out_wide);
            }
          } else if (whole) {
            float* to = static_cast<float*>(p.out) + out0;
#pragma unroll
            for (int u = 0; u < kCols; u += 8) {
              uint32_t y[8];
#pragma unroll
              for (int v = 0; v < 8; ++v) y[v] = o[u / 32][u % 32 + v];
              store_sector(to + u, y, p.out_wide);
            }
          }
          // Non-finite V elements of nodes this row sees (rare) are added to what was
          // stored: the sum of a finite number and one of them is the same after its
          // rounding to bf16.
          for (unsigned long long h = hit; h; h &= h - 1) {
            const int at = base + __ffsll(h) - 1;
            const int id = __ldg(p.block_tables + size_t(seq) * p.max_blocks_per_seq + at / 16);
            const uint16_t* row = static_cast<const uint16_t*>(p.v_pool) + col0 +
                                  ((int64_t(id) * 16 + at % 16) * p.kv_heads + kvh) * D;
#pragma unroll 1
            for (int u = 0; u < kCols; ++u) {
              const uint32_t v = row[u];
              if ((v & 0x7f80u) != 0x7f80u) continue;
              const float add = __uint_as_float(v << 16);
              if (!whole) {
                const size_t tile = (size_t(blockIdx.x) * 2 + (k == 0 ? 0 : 1)) * TILES +
                                    (TILES == 2 ? w : 0);
                p.part_o[((tile * (D / 4) + (col0 + u) / 4) * kTrRows + r) * 4 + u % 4] += add;
              } else if (p.out_bf16) {
                __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.out) + out0 + u;
                *y = __float2bfloat16(__bfloat162float(*y) + add);
              } else {
                static_cast<float*>(p.out)[out0 + u] += add;
              }
            }
          }
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) tr_abort(abort_flag);
  }
  }  // count > 0

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTrTmemCols);
  }
}

// Joins the pieces of the items that were cut between CTAs.  Block (b, y):
// rows 32 y .. of the item in which CTA b + 1's range starts, if the range of
// an earlier CTA does not start inside the same item (each cut item then has
// one b); its pieces are CTA b's last one and the first ones of b + 1, b + 2,
// ... while they are of the item.  out = sum 2^(lse_i - lse) o_i; lane = row,
// a warp takes an eighth of the quads of columns, as the pieces are laid out,
// and the rows leave through shared memory.
constexpr int kTrMergeThreads = 256;

template <int D, int G, int TILES>
__global__ void __launch_bounds__(kTrMergeThreads)
tree_merge_kernel(const TreeParams p, int ctas) {
  constexpr int kQuads = D / 4 / 8;  // per warp
  __shared__ __align__(16) float rows_out[32][D + 4];
  const int b = blockIdx.x + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  // lane i: CTA b - 1 + i; the CTAs b, b + 1, ... whose ranges start in the item
  TreeStart at{-1, 0, 0, 0, 0, 0, {0, 0}};
  if (b - 1 + lane < ctas) at = p.start[b - 1 + lane];
  const int seq = __shfl_sync(0xffffffffu, at.seq, 1);
  const int item = __shfl_sync(0xffffffffu, at.item, 1);
  if (seq < 0 || __shfl_sync(0xffffffffu, at.tile, 1) == 0) return;
  const bool mine = at.seq == seq && at.item == item;
  unsigned vote = __ballot_sync(0xffffffffu, mine);
  const bool same = vote & 1u;  // CTA b - 1's range starts in the item, too
  if (same && __shfl_sync(0xffffffffu, at.tile, 0) > 0) return;
  const int qs = __shfl_sync(0xffffffffu, at.qs, 1);
  const int nodes = __shfl_sync(0xffffffffu, at.n, 1);
  const int groups = __shfl_sync(0xffffffffu, at.groups, 1);
  const int kvh = item / groups, group = item - kvh * groups;
  const int node0 = group * TILES * (kTrRows / G);
  const int rows = min((nodes - node0) * G, TILES * kTrRows) - int(blockIdx.y) * 32;
  if (rows <= 0) return;  // uniform over the block, as all returns are
  vote |= 1u;
  int parts = vote == 0xffffffffu ? 32 : __ffs(~vote) - 1;
  while (parts % 32 == 0) {  // more than the lanes look at at a time
    const int c = b - 1 + parts + lane;
    const bool more = c < ctas && p.start[c].seq == seq && p.start[c].item == item;
    vote = __ballot_sync(0xffffffffu, more);
    if (vote == 0) break;
    parts += vote == 0xffffffffu ? 32 : __ffs(~vote) - 1;
  }
  // piece i's tile of 128 rows in the workspace, and this lane's row of it
  const int tile = blockIdx.y / 4, r = (blockIdx.y % 4) * 32 + lane;
  auto tile_of = [&](int i) {
    const size_t slot = i == 0 ? size_t(b - 1) * 2 + (same ? 0 : 1) : size_t(b + i - 1) * 2;
    return slot * TILES + tile;
  };
  float4 acc[kQuads];
#pragma unroll
  for (int z = 0; z < kQuads; ++z) acc[z] = make_float4(0.f, 0.f, 0.f, 0.f);
  float big = -INFINITY, tot = 0.f;
  // Several pieces' loads at a time, those beyond the last as pieces without
  // weight.  More at a time take registers, and with them the blocks that an SM
  // holds: us with 2 / 3 / 4 / 8, heads of 128: 1 x 500, 8 nodes 11.8 / 11.7 / 11.7 /
  // 11.7, 64 x 700, 4 nodes 44.5 / 43.6 / 43.6 / 43.3, 32 x 1000, 16 nodes 36.4 / 37.3 /
  // 37.4 / 39.4, 16 x 4000, 64 nodes 112.5 / 115.4 / 114.7 / 121.5; with 1 / 4 / 8, heads
  // of 64: 1 x 30000, 27 nodes 34.7 / 28.9 / 28.8.
  constexpr int kAtOnce = D == 64 ? 8 : 2;
  if (lane < rows) {
#pragma unroll 1
    for (int i = 0; i < parts; i += kAtOnce) {
      float lse[kAtOnce];
      float4 x[kAtOnce][kQuads];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const size_t t = tile_of(min(i + u, parts - 1));
        const float4* o = reinterpret_cast<const float4*>(p.part_o) +
                          (t * (D / 4) + warp * kQuads) * kTrRows + r;
        lse[u] = -INFINITY;
#pragma unroll
        for (int z = 0; z < kQuads; ++z) x[u][z] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i + u < parts) {
          lse[u] = __ldg(p.part_lse + t * kTrRows + r);
#pragma unroll
          for (int z = 0; z < kQuads; ++z) x[u][z] = __ldg(o + z * kTrRows);
        }
      }
      float now = big;
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) now = fmaxf(now, lse[u]);
      const float ref = now == -INFINITY ? 0.f : now;
      const float fade = ex2(big - ref);
      big = now;
      tot *= fade;
#pragma unroll
      for (int z = 0; z < kQuads; ++z) {
        acc[z].x *= fade;
        acc[z].y *= fade;
        acc[z].z *= fade;
        acc[z].w *= fade;
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const float wgt = ex2(lse[u] - ref);
        tot += wgt;  // a piece in which the row saw nothing weighs 0 (its row is zeros)
#pragma unroll
        for (int z = 0; z < kQuads; ++z) {
          acc[z].x += x[u][z].x * wgt;
          acc[z].y += x[u][z].y * wgt;
          acc[z].z += x[u][z].z * wgt;
          acc[z].w += x[u][z].w * wgt;
        }
      }
    }
  }
  const float inv = tot != 0.f ? 1.f / tot : 0.f;
#pragma unroll
  for (int z = 0; z < kQuads; ++z)
    *reinterpret_cast<float4*>(&rows_out[lane][(warp * kQuads + z) * 4]) =
        make_float4(acc[z].x * inv, acc[z].y * inv, acc[z].z * inv, acc[z].w * inv);
  __syncthreads();
  for (int k = threadIdx.x; k < 32 * (D / 4); k += kTrMergeThreads) {
    const int row = k / (D / 4), col = (k % (D / 4)) * 4;
    if (row >= rows) break;
    const float4 y = *reinterpret_cast<const float4*>(&rows_out[row][col]);
    const int rr = int(blockIdx.y) * 32 + row;
    const size_t to =
        ((size_t(qs) + node0 + rr / G) * p.q_heads + size_t(kvh) * G + rr % G) * D + col;
    if (p.out_bf16)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + to) =
          make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to) = y;
  }
}

cudaError_t tree_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_tree_error);
}

unsigned read_tree_error(bool clear) {
  unsigned word = 0;
  if (cudaMemcpyFromSymbol(&word, g_tree_error, sizeof(word)) != cudaSuccess) return ~0u;
  if (clear) {
    const unsigned zero = 0;
    if (cudaMemcpyToSymbol(g_tree_error, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  }
  return word;
}

int tree_tile_rows() { return kTrRows; }
int tree_tile_keys() { return kTrKeys; }
int tree_places(int tiles) { return tiles + kTrSlack; }

template <int D, int G, int TILES>
static cudaError_t launch_tree_t(const TreeParams& p, int ctas, const CUtensorMap* tq,
                                 const CUtensorMap* tk, const CUtensorMap* tv,
                                 cudaStream_t stream) {
  using T = TreeSmem<D, TILES>;
  static std::atomic<int> attr_done[kAttrMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kAttrMaxDevices || !attr_done[dev].load(std::memory_order_acquire)) {
    // the split of the registers draws on what the launch allots: an increase
    // beyond it would wait forever
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, paged_tree_kernel<D, G, TILES>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * kTrThreads < 256 * kTrRegsSoftmax + (kTrThreads - 256) * kTrRegsIssue)
      return cudaErrorInvalidConfiguration;
    e = set_smem_limit_once(paged_tree_kernel<D, G, TILES>, T::kSmemBytes, attr_done);
    if (e != cudaSuccess) return e;
  }
  e = launch_after_previous(paged_tree_kernel<D, G, TILES>, dim3(ctas), dim3(kTrThreads),
                            T::kSmemBytes, stream, *tq, *tk, *tv, p);
  if (e != cudaSuccess || ctas < 2) return e;
  const int rows = std::min(p.max_q_len * G, TILES * kTrRows);
  return launch_after_previous(tree_merge_kernel<D, G, TILES>,
                               dim3(ctas - 1, (rows + 31) / 32), dim3(kTrMergeThreads), 0, stream,
                               p, ctas);
}

template <int D, int TILES>
static cudaError_t launch_tree_g(const TreeParams& p, int ctas, int group, const CUtensorMap* tq,
                                 const CUtensorMap* tk, const CUtensorMap* tv,
                                 cudaStream_t stream) {
  switch (group) {
    case 1: return launch_tree_t<D, 1, TILES>(p, ctas, tq, tk, tv, stream);
    case 2: return launch_tree_t<D, 2, TILES>(p, ctas, tq, tk, tv, stream);
    case 4: return launch_tree_t<D, 4, TILES>(p, ctas, tq, tk, tv, stream);
    case 8: return launch_tree_t<D, 8, TILES>(p, ctas, tq, tk, tv, stream);
    case 16: return launch_tree_t<D, 16, TILES>(p, ctas, tq, tk, tv, stream);
    default: return cudaErrorInvalidValue;
  }
}

int tree_tiles(int group, int max_q_len) { return group * max_q_len <= kTrRows ? 1 : 2; }

cudaError_t launch_paged_tree(const TreeArgs& a, const CUtensorMap* tq, const CUtensorMap* tk,
                              const CUtensorMap* tv, cudaStream_t stream) {
  TreeParams p;
  p.q_start = a.q_start;
  p.tree_mask = reinterpret_cast<const unsigned long long*>(a.tree_mask);
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.v_pool = a.v_cache;
  p.out = a.out;
  p.out_bf16 = a.out_bf16 ? 1 : 0;
  p.out_wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
  p.part_o = a.part_o;
  p.part_lse = a.part_lse;
  p.start = static_cast<TreeStart*>(a.start);
  p.num_seqs = a.num_seqs;
  p.total_q = a.total_q;
  p.max_q_len = a.max_q_len;
  p.q_heads = a.q_heads;
  p.kv_heads = a.kv_heads;
  // the most parts that divide the KV heads and leave at most a 20th of the CTAs over
  p.lanes = a.kv_heads;
  while (p.lanes > 1 && (a.kv_heads % p.lanes != 0 || a.ctas % p.lanes * 20 > a.ctas)) --p.lanes;
  p.num_blocks = a.num_blocks;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.scale_log2 = a.scale_log2;
  const int group = a.q_heads / a.kv_heads;
  const bool one = tree_tiles(group, a.max_q_len) == 1;
  if (a.d_head == 128)
    return one ? launch_tree_g<128, 1>(p, a.ctas, group, tq, tk, tv, stream)
               : launch_tree_g<128, 2>(p, a.ctas, group, tq, tk, tv, stream);
  if (a.d_head == 64)
    return one ? launch_tree_g<64, 1>(p, a.ctas, group, tq, tk, tv, stream)
               : launch_tree_g<64, 2>(p, a.ctas, group, tq, tk, tv, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pkv
