// Paged decode attention over the block-scaled FP8 cache: one query per
// sequence, K = k_scales[block][head] * e4m3(code), V alike.
//
// Mathematics, per KV head with its group of G query heads, in log2 units:
//   x_j = (q . code_j) * scale log2(e) * k_scale(block of j)
//   m = max x,  l = sum 2^(x - m),  O = sum 2^(x - m) v_scale code_v / l
// A block's scales are constants of 16 keys, so they join the arithmetic where
// a whole block is one factor: K's in the factor that scores have anyway, V's
// in the weights on their way to the second product.  The weights enter that
// product as f16, so O has a running maximum of its own,
//   dv = max ((x - m) + floor(log2 v_scale)),
// and is kept in units of 2^(m + dv - 14): a weight v_scale 2^(x - m - dv + 14) is below
// 2^15 for every row (f16 ends at 2^16), and a block counts by what it gives to the row,
// whatever scales blocks have to which the row pays no heed.  What is below 2^-39 of a
// row's largest is lost, the rest within 2^-11 of itself or 2^-39 of the largest (with
// weights up to 2 the tail of a long context, 10^5 keys of weights below 2^-25, was lost
// as a whole).  dv is kept beside m and not added to it: a score of 2^31 would swallow
// it.  For the same reason the pieces of a pair meet as (m, l) and not as m + log2 l: rows
// of equal scores are means of their values however large the scores.  Queries are f16
// after an exact power of two that brings a row outside [2^-6, 2^15) into it.
//
// Bound by HBM: every code is read once, 4 flops for each byte and query head.
// A warp owns a ring of pages (K and V of one KV head, fetched by TMA) and runs
// the f16 warp MMAs on the converted codes; the page arithmetic is that of the
// per-pool decode (pkv_decode_fp8_body.cuh), with the two factors.
//
// Three splits of the work:
//  * cluster: a (sequence, KV head) pair belongs to a cluster of 1 to 8 CTAs
//    of four warps, whose warps take the pair's pages in turn; the warps'
//    results meet in shared memory and the CTAs' over distributed shared
//    memory.  One launch, no workspace: for batches whose pages fit one wave.
//  * pairs: each warp takes a (sequence, KV head) pair whole.  One launch: for
//    more pairs than clusters of one CTA run at once, of up to 32 pages each.
//  * flat: the pages of all sequences laid end to end are cut into equal
//    ranges, one for each group of Hkv warps of a grid of one CTA per SM (as in
//    paged_decode_flat.cu); a second kernel joins the pieces of the pairs that
//    were cut.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "pkv_decode_flat_body.cuh"
#include "pkv_internal.h"

namespace pkv {

// The lane of a converged warp that issues its copies (always the same one).
__device__ __forceinline__ bool elect_lane() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

struct BsDecodeParams {
  DecodeParams d;  // scale_log2 without the K scale; out_scale is not used
  const float* k_scales;
  const float* v_scales;
  float2* part_ml;  // a piece's maximum and sum (d.part_o: its normalised rows)
  int max_blocks;   // pages attended per sequence at most
};

template <int D>
struct BsPage {
  static constexpr int kTileBytes = kBlockTokens * D;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = D == 128 ? 4 : 8;  // 16 KB a warp
  static constexpr int kRingBytes = kStages * kStageBytes;
  // byte address of 16-byte chunk c of row r: rows of 128 (64) bytes, written
  // by TMA with the 128- (64-) byte swizzle
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  }
};

// Running state of one warp (layout of the accumulators as in F8Acc).
template <int D, int G>
struct BsAcc {
  static constexpr int NH = (G + 7) / 8;
  static constexpr int MT = D / 16;
  static constexpr float kUp = 0x1p14f;
  float o[NH][MT][4];
  float m[NH][2], l[NH][2];
  float dv[NH][2];    // O is in units of 2^(m + dv) / kUp
  float qmul[NH][2];  // what the queries were divided by, times the softmax scale
  uint32_t qf[NH][MT][2];

  // The queries of rows row0 .. row0 + G - 1, in the order in which the K
  // fragments arrive (see pkv_decode_fp8_body.cuh), and an empty state.
  __device__ __forceinline__ void start(const __nv_bfloat16* q, size_t row0, float scale_log2,
                                        int lane) {
    const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      const int head = 8 * nh + gid;
      uint2 w[MT];
      uint32_t top = 0;
#pragma unroll
      for (int kk = 0; kk < MT; ++kk) {
        w[kk] = head < G ? __ldg(reinterpret_cast<const uint2*>(q + (row0 + head) * D + kk * 16 +
                                                                4 * tig))
                         : make_uint2(0, 0);
        top = __vmaxu2(__vmaxu2(top, w[kk].x & 0x7fff7fffu), w[kk].y & 0x7fff7fffu);
      }
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // bf16 exponent of the largest element; 127 + [-6, 14] stays as it is
      const int e = int(max(top & 0xffffu, top >> 16) >> 7);
      const int shift = e < 121 || e > 141 ? min(max(e, 1), 253) - 127 : 0;
      const float inv = __uint_as_float(uint32_t(127 - shift) << 23);  // 2^-shift, shift <= 126: normal
      const float mul = __uint_as_float(uint32_t(127 + shift) << 23) * scale_log2;
#pragma unroll
      for (int kk = 0; kk < MT; ++kk) {
        qf[nh][kk][0] = pack_f16x2(bf16_lo_to_f32(w[kk].x) * inv, bf16_hi_to_f32(w[kk].x) * inv);
        qf[nh][kk][1] = pack_f16x2(bf16_lo_to_f32(w[kk].y) * inv, bf16_hi_to_f32(w[kk].y) * inv);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        qmul[nh][c] = __shfl_sync(0xffffffffu, mul, (2 * tig + c) * 4);
        m[nh][c] = -INFINITY;
        l[nh][c] = dv[nh][c] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) o[nh][mt][0] = o[nh][mt][1] = o[nh][mt][2] = o[nh][mt][3] = 0.f;
    }
  }
  // an element of O over `l`, in the weights' units (factor by factor: their product may
  // be a number of few bits where the result is not)
  __device__ __forceinline__ float value(int nh, int mt, int e, float inv_l, float unit) const {
    return o[nh][mt][e] * ((1.f / kUp) * inv_l) * unit;
  }
  // O's unit, kUp aside, over the weights' (an empty state's O is 0)
  __device__ __forceinline__ float unit(int nh, int c) const {
    return m[nh][c] == -INFINITY ? 0.f : ex2(dv[nh][c]);
  }

  __device__ __forceinline__ void sum_l() {
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[nh][c] += __shfl_xor_sync(0xffffffffu, l[nh][c], 4);
        l[nh][c] += __shfl_xor_sync(0xffffffffu, l[nh][c], 8);
        l[nh][c] += __shfl_xor_sync(0xffffffffu, l[nh][c], 16);
      }
  }
};

// FULL: every page lies within the sequence, and nothing is masked.
// NP landed pages: page i at kbase[i], its first token tok0[i], its scales
// ks[i] and vs[i]; the sequence ends at `len`.
template <int D, int G, int NP, bool FULL>
__device__ __forceinline__ void bs_pages_as(BsAcc<D, G>& A, const uint32_t (&kbase)[NP],
                                         const int (&tok0)[NP], const float (&ks)[NP],
                                         const float (&vs)[NP], int len, int lane) {
  using T = BsPage<D>;
  constexpr int NH = BsAcc<D, G>::NH;
  constexpr int MT = BsAcc<D, G>::MT;
  const int gid = lane >> 2, tig = lane & 3;
  const int mi = lane >> 3, mr = lane & 7;
  const int k_tok = (mi >> 1) * 8 + mr;
  const int v_tok = (mi & 1) * 8 + mr;

  // S^T = K Q^T, even and odd k-steps accumulated separately
  float s[NP][NH][4], s_odd[NP][NH][4];
#pragma unroll
  for (int pg = 0; pg < NP; ++pg)
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[pg][nh][e] = s_odd[pg][nh][e] = 0.f;
#pragma unroll
  for (int kp = 0; kp < D / 32; ++kp) {
#pragma unroll
    for (int pg = 0; pg < NP; ++pg) {
      uint32_t r0, r1, r2, r3;
      ldsm_x4(kbase[pg] + T::at(k_tok, 2 * kp + (mi & 1)), r0, r1, r2, r3);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a0, a1, a2, a3;
        e4m3x4_to_f16x2x2(h ? r1 : r0, a0, a2);
        e4m3x4_to_f16x2x2(h ? r3 : r2, a1, a3);
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
          mma_f16_16816(h ? s_odd[pg][nh] : s[pg][nh], a0, a1, a2, a3, A.qf[nh][2 * kp + h][0],
                        A.qf[nh][2 * kp + h][1]);
      }
    }
  }

  float lv[NP];  // exponents of V's scales, no less than a normal number's
#pragma unroll
  for (int pg = 0; pg < NP; ++pg)
    lv[pg] = float(max(int(__float_as_uint(vs[pg]) >> 23), 1) - 127);

  // online softmax per head column, in the log2 domain
  bool k0_in[NP], k1_in[NP];
#pragma unroll
  for (int pg = 0; pg < NP; ++pg) {
    k0_in[pg] = tok0[pg] + gid < len;
    k1_in[pg] = tok0[pg] + gid + 8 < len;
  }
  uint32_t pb[NP][NH][2];
  float beta[NH][2];
  bool all_same = true;
#pragma unroll
  for (int nh = 0; nh < NH; ++nh) {
    float pr[NP][4], w[NP][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float x0[NP], x1[NP], top[NP];
#pragma unroll
      for (int pg = 0; pg < NP; ++pg) {
        const float f = ks[pg] * A.qmul[nh][c];
        x0[pg] = FULL || k0_in[pg] ? (s[pg][nh][c] + s_odd[pg][nh][c]) * f : -INFINITY;
        x1[pg] = FULL || k1_in[pg] ? (s[pg][nh][c + 2] + s_odd[pg][nh][c + 2]) * f : -INFINITY;
        top[pg] = fmaxf(x0[pg], x1[pg]);
      }
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1)
#pragma unroll
        for (int pg = 0; pg < NP; ++pg)
          top[pg] = fmaxf(top[pg], __shfl_xor_sync(0xffffffffu, top[pg], o));
      float mn = A.m[nh][c];
#pragma unroll
      for (int pg = 0; pg < NP; ++pg) mn = fmaxf(mn, top[pg]);
      const float fall = A.m[nh][c] - mn, dv = A.dv[nh][c] + fall;  // (-inf at first)
      float dvn = dv;
#pragma unroll
      for (int pg = 0; pg < NP; ++pg) dvn = fmaxf(dvn, (top[pg] - mn) + lv[pg]);
      const float alpha = ex2(fall);
      beta[nh][c] = ex2(dv - dvn);
      all_same = all_same && dv == dvn;
      A.m[nh][c] = mn;
      A.dv[nh][c] = dvn;
      // (bounded: a block whose weights are below 2^-112 may have a larger factor, past
      // float32 even)
      const float unit = ex2(-dvn);
#pragma unroll
      for (int pg = 0; pg < NP; ++pg) {
        const float f = vs[pg] * unit;
        w[pg][c] = (f > 0x1p112f ? 0x1p112f : f) * A.kUp;
      }
      float add = 0.f;
#pragma unroll
      for (int pg = 0; pg < NP; ++pg) {
        pr[pg][c] = ex2(x0[pg] - mn);
        pr[pg][c + 2] = ex2(x1[pg] - mn);
        add += pr[pg][c] + pr[pg][c + 2];
      }
      A.l[nh][c] = A.l[nh][c] * alpha + add;
    }
    // P^T as the B operand: (key, two heads) per lane -> (two keys, head)
#pragma unroll
    for (int pg = 0; pg < NP; ++pg) {
      pb[pg][nh][0] = movmatrix_trans(pack_f16x2(pr[pg][0] * w[pg][0], pr[pg][1] * w[pg][1]));
      pb[pg][nh][1] = movmatrix_trans(pack_f16x2(pr[pg][2] * w[pg][0], pr[pg][3] * w[pg][1]));
    }
  }
  if (!__all_sync(0xffffffffu, all_same)) {
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      const float a0 = beta[nh][0], a1 = beta[nh][1];  // 0 at first
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        A.o[nh][mt][0] *= a0;
        A.o[nh][mt][1] *= a1;
        A.o[nh][mt][2] *= a0;
        A.o[nh][mt][3] *= a1;
      }
    }
  }

  // O^T += V^T P^T; codes of rows past the length may be NaN: zeroed
  uint32_t vm0[NP], vm1[NP];
#pragma unroll
  for (int pg = 0; pg < NP; ++pg) {
    vm0[pg] = vm1[pg] = 0xffffffffu;
    if (!FULL && tok0[pg] + kBlockTokens > len) {
      const int k0 = tok0[pg] + 2 * tig;
      vm0[pg] = (k0 < len ? 0x0000ffffu : 0u) | (k0 + 1 < len ? 0xffff0000u : 0u);
      vm1[pg] = (k0 + 8 < len ? 0x0000ffffu : 0u) | (k0 + 9 < len ? 0xffff0000u : 0u);
    }
  }
#pragma unroll
  for (int cp = 0; cp < D / 32; ++cp) {
#pragma unroll
    for (int pg = 0; pg < NP; ++pg) {
      uint32_t r0, r1, r2, r3;
      ldsm_x4_trans(kbase[pg] + T::kTileBytes + T::at(v_tok, 2 * cp + (mi >> 1)), r0, r1, r2, r3);
      if constexpr (!FULL) {
        r0 &= vm0[pg];
        r1 &= vm1[pg];
        r2 &= vm0[pg];
        r3 &= vm1[pg];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a0, a1, a2, a3;
        e4m3x4_to_f16x2x2(__byte_perm(h ? r2 : r0, 0u, 0x3120), a0, a1);
        e4m3x4_to_f16x2x2(__byte_perm(h ? r3 : r1, 0u, 0x3120), a2, a3);
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
          mma_f16_16816(A.o[nh][2 * cp + h], a0, a1, a2, a3, pb[pg][nh][0], pb[pg][nh][1]);
      }
    }
  }
}

template <int D, int G, int NP>
__device__ __forceinline__ void bs_pages(BsAcc<D, G>& A, const uint32_t (&kbase)[NP],
                                         const int (&tok0)[NP], const float (&ks)[NP],
                                         const float (&vs)[NP], int len, int lane) {
  if (NP == 2 && tok0[NP - 1] + kBlockTokens <= len)  // the last one is the furthest
    bs_pages_as<D, G, NP, true>(A, kbase, tok0, ks, vs, len, lane);
  else
    bs_pages_as<D, G, NP, false>(A, kbase, tok0, ks, vs, len, lane);
}

// One page's two boxes into a ring stage, by the warp as a whole: the copies'
// operands are then values of the warp.  Issued from a branch on the lane number
// they take 390 cycles a page, so 290 (24 x 2500 tokens, heads of 64: 10.0 us, 9.2).
template <int D>
__device__ __forceinline__ void bs_issue(uint32_t dst, uint32_t bar, const CUtensorMap& tk,
                                         const CUtensorMap& tv, int head, int id) {
  if (elect_lane()) {
    mbar_arrive_expect_tx(bar, BsPage<D>::kStageBytes);
    tma_load_4d(dst, &tk, bar, 0, head, 0, id);
    tma_load_4d(dst + BsPage<D>::kTileBytes, &tv, bar, 0, head, 0, id);
  }
}

// A warp's `cnt` pages, the i-th at block page0 + i step of the sequence, lane i
// holding its id and scales: attended by the queries of rows row0 on.
template <int D, int G>
__device__ __forceinline__ void bs_walk(BsAcc<D, G>& acc, uint32_t ring, uint32_t bars,
                                        const CUtensorMap& tmap_k, const CUtensorMap& tmap_v,
                                        const DecodeParams& p, size_t row0, int kvh, int id,
                                        float ks, float vs, int cnt, int page0, int step, int len,
                                        int lane) {
  using T = BsPage<D>;
  constexpr int kStages = T::kStages;
  constexpr unsigned kFull = 0xffffffffu;
  auto issue = [&](int i) {  // warp-wide
    const int st = i % kStages;
    bs_issue<D>(ring + st * T::kStageBytes, bars + st * 8, tmap_k, tmap_v, kvh,
                __shfl_sync(kFull, id, i));
  };
  for (int i = 0; i < cnt && i < kStages; ++i) issue(i);
  int issued = min(cnt, kStages);

  acc.start(p.q, row0, p.scale_log2, lane);
  bool failed = false;
  int i = 0;
  while (i < cnt) {
    const bool two = i + 1 < cnt;
    bool landed = mbar_wait_bounded(bars + (i % kStages) * 8, (i / kStages) & 1);
    if (two && landed)
      landed = mbar_wait_bounded(bars + ((i + 1) % kStages) * 8, ((i + 1) / kStages) & 1);
    if (!__all_sync(kFull, landed)) {
      failed = true;
      break;
    }
    const uint32_t b0 = ring + (i % kStages) * T::kStageBytes;
    const int t0 = (page0 + i * step) * kBlockTokens;
    const float ks0 = __shfl_sync(kFull, ks, i), vs0 = __shfl_sync(kFull, vs, i);
    if (two) {
      const uint32_t kb[2] = {b0, ring + ((i + 1) % kStages) * T::kStageBytes};
      const int tk[2] = {t0, t0 + step * kBlockTokens};
      const float k2[2] = {ks0, __shfl_sync(kFull, ks, i + 1)};
      const float v2[2] = {vs0, __shfl_sync(kFull, vs, i + 1)};
      bs_pages<D, G, 2>(acc, kb, tk, k2, v2, len, lane);
    } else {
      const uint32_t kb[1] = {b0};
      const int tk[1] = {t0};
      const float k1[1] = {ks0}, v1[1] = {vs0};
      bs_pages<D, G, 1>(acc, kb, tk, k1, v1, len, lane);
    }
    __syncwarp();
    const int n = two ? 2 : 1;
    for (int j = i; j < i + n; ++j)
      if (j + kStages < cnt) {
        issue(j + kStages);
        ++issued;
      }
    i += n;
  }
  if (failed) {
    if (lane == 0) {
      atomicOr(&g_decode_error, kErrWaitTimeout);
      for (int k = i; k < issued; ++k)
        (void)mbar_wait_bounded(bars + (k % kStages) * 8, (k / kStages) & 1);
    }
    __syncwarp();
  }
}

// ------------------------------------------------------------ cluster split
constexpr int kBsClWarps = 4;
constexpr int kBsClMaxCtas = 8;    // per cluster: the portable limit
constexpr int kBsClMaxPages = 32;  // per warp: one lane holds each page's id and scales

template <int D, int G>
struct BsCl {
  static constexpr int kRings = kBsClWarps * BsPage<D>::kRingBytes;
  static constexpr int kBarOff = kRings;
  static constexpr int kOutOff = kBarOff + kBsClWarps * BsPage<D>::kStages * 8;
  static constexpr int kRowFloats = G * D + 2 * G;  // O, then each row's m and l
  static constexpr int kSmemBytes = kOutOff + kRowFloats * 4 + 1024;
  static_assert(kRowFloats * 4 <= BsPage<D>::kRingBytes, "a warp's result fits its ring");
};

template <int D, int G>
__global__ void __launch_bounds__(kBsClWarps * 32, 3)
decode_block_scaled_cluster_kernel(const __grid_constant__ CUtensorMap tmap_k,
                                   const __grid_constant__ CUtensorMap tmap_v,
                                   const BsDecodeParams bp) {
  using T = BsPage<D>;
  using L = BsCl<D, G>;
  constexpr int kStages = T::kStages;
  constexpr unsigned kFull = 0xffffffffu;
  const DecodeParams& p = bp.d;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(kFull, int(threadIdx.x >> 5), 0);  // a value of the warp
  const int gid = lane >> 2, tig = lane & 3;
  const int pair = blockIdx.x / C;
  const int seq = pair / p.kv_heads, kvh = pair - seq * p.kv_heads;
  const uint32_t ring = smem_u32(smem + warp * T::kRingBytes);
  const uint32_t bars = smem_u32(smem + L::kBarOff) + warp * kStages * 8;

  if (lane == 0) {
    for (int st = 0; st < kStages; ++st) mbar_init(bars + st * 8, 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
  }
  __syncwarp();
  griddep_wait();
  griddep_launch_dependents();

  // page i of this warp: the pair's page (i C + rank) W + warp
  const int page0 = rank * kBsClWarps + warp, step = C * kBsClWarps;
  int id = 0;
  const int mine = page0 + lane * step;
  if (mine < bp.max_blocks) id = __ldg(p.block_tables + size_t(seq) * p.max_blocks_per_seq + mine);
  bool bad;
  const int raw = __ldg(p.context_lens + seq);
  const int nblk = flat_pages(raw, bp.max_blocks, bad);
  if (bad && kvh == 0 && rank == 0 && threadIdx.x == 0) atomicOr(&g_decode_error, kErrBadContext);
  const int len = raw < 0 ? 0 : min(raw, nblk * kBlockTokens);
  const int cnt = nblk > page0 ? (nblk - page0 + step - 1) / step : 0;
  float ks = 0.f, vs = 0.f;
  if (lane < cnt) {
    if (id >= 0 && id < p.num_blocks) {
      ks = __ldg(bp.k_scales + size_t(id) * p.kv_heads + kvh);
      vs = __ldg(bp.v_scales + size_t(id) * p.kv_heads + kvh);
    } else {
      atomicOr(&g_decode_error, kErrBadBlockId);
    }
  }
  BsAcc<D, G> acc;
  const size_t row0 = size_t(seq) * p.q_heads + size_t(kvh) * G;
  bs_walk<D, G>(acc, ring, bars, tmap_k, tmap_v, p, row0, kvh, id, ks, vs, cnt, page0, step, len,
                lane);
  acc.sum_l();

  // the warp's result over its own ring: O in the weights' unit, m, l
  float* mo = reinterpret_cast<float*>(smem + warp * T::kRingBytes);
#pragma unroll
  for (int nh = 0; nh < BsAcc<D, G>::NH; ++nh)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int head = 8 * nh + 2 * tig + c;
      if (head >= G) continue;
      const float unit = acc.unit(nh, c);
#pragma unroll
      for (int mt = 0; mt < BsAcc<D, G>::MT; ++mt)
        *reinterpret_cast<float2*>(mo + head * D + 16 * mt + 2 * gid) =
            make_float2(acc.value(nh, mt, c, 1.f, unit), acc.value(nh, mt, c + 2, 1.f, unit));
      if (gid == 0) {
        reinterpret_cast<float2*>(mo + G * D)[head] = make_float2(acc.m[nh][c], acc.l[nh][c]);
      }
    }
  __syncthreads();
  // the CTA's: normalised O, m and l (0: no key)
  float* part = reinterpret_cast<float*>(smem + L::kOutOff);
  for (int x = threadIdx.x * 4; x < G * D; x += kBsClWarps * 32 * 4) {
    const int row = x / D;
    float big = -INFINITY;
#pragma unroll
    for (int w = 0; w < kBsClWarps; ++w)
      big = fmaxf(big, reinterpret_cast<const float2*>(smem + w * T::kRingBytes + G * D * 4)[row].x);
    float tot = 0.f;
    float4 val = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kBsClWarps; ++w) {
      const float* wo = reinterpret_cast<const float*>(smem + w * T::kRingBytes);
      const float2 ml = reinterpret_cast<const float2*>(wo + G * D)[row];
      const float wgt = ml.x == -INFINITY ? 0.f : ex2(ml.x - big);
      const float4 o = *reinterpret_cast<const float4*>(wo + x);
      tot += ml.y * wgt;
      val.x += o.x * wgt;
      val.y += o.y * wgt;
      val.z += o.z * wgt;
      val.w += o.w * wgt;
    }
    const float inv = big == -INFINITY && tot == 0.f ? 0.f : 1.f / tot;
    *reinterpret_cast<float4*>(part + x) =
        make_float4(val.x * inv, val.y * inv, val.z * inv, val.w * inv);
    if (x == row * D) reinterpret_cast<float2*>(part + G * D)[row] = make_float2(big, tot);
  }
  if (C == 1) {
    __syncthreads();
    for (int x = threadIdx.x; x < G * D; x += kBsClWarps * 32) store_out(p, row0 * D + x, part[x]);
    return;
  }
  cluster.sync();
  // each CTA writes its share of the rows' elements
  const int share = G * D / C;  // a multiple of 8: G D >= 64, C <= 8
  for (int x = rank * share + int(threadIdx.x); x < (rank + 1) * share; x += kBsClWarps * 32) {
    const int row = x / D;
    float2 ml[kBsClMaxCtas];
    float o[kBsClMaxCtas];
#pragma unroll
    for (int c = 0; c < kBsClMaxCtas; ++c) {
      if (c < C) {
        const float* other = cluster.map_shared_rank(part, c);
        ml[c] = reinterpret_cast<const float2*>(other + G * D)[row];
        o[c] = other[x];
      } else {
        ml[c] = make_float2(-INFINITY, 0.f);
        o[c] = 0.f;
      }
    }
    float big = -INFINITY;
#pragma unroll
    for (int c = 0; c < kBsClMaxCtas; ++c) big = fmaxf(big, ml[c].x);
    float tot = 0.f, val = 0.f;
#pragma unroll
    for (int c = 0; c < kBsClMaxCtas; ++c) {
      const float wgt = ml[c].y == 0.f ? 0.f : ml[c].y * ex2(ml[c].x - big);
      tot += wgt;
      val += o[c] * wgt;
    }
    store_out(p, row0 * D + x, tot == 0.f ? 0.f : val / tot);
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

// -------------------------------------------------------- a pair to each warp
// The four warps of a CTA take four pairs, whole and by themselves: no join, no
// second launch, and CTAs are handed out as others end (256 contexts of up to 200
// tokens, 64 heads of 128 on 8: 15.3 us, 27.2 with the flat split; 254 of one token,
// 128 / 8 of 64: 5.8, 16.9; 256 of 500, 64 / 8 of 128: 57, 62).  From where it begins,
// at 464 pairs, to 2432, of 2 to 32 pages, full and ragged, heads of 128 in groups of 8
// and of 1 and of 64 in groups of 2, it takes 0.27 to 1.02 of the flat split's time (464
// pairs of 32 pages, 64 / 8 of 128: 16.8 us, 21.1), but for heads of 64 with 32 pages
// at some counts (1216 pairs 26.6 us, 25.2; 2432 43.3, 39.4).  One long context
// among short ones is what the flat split does better (15 of 30 tokens and one of
// 500, 32 / 32 heads of 128: 9.5 against 13.0).
template <int D, int G>
__global__ void __launch_bounds__(kBsClWarps * 32, 3)
decode_block_scaled_pairs_kernel(const __grid_constant__ CUtensorMap tmap_k,
                                 const __grid_constant__ CUtensorMap tmap_v,
                                 const BsDecodeParams bp, int pairs) {
  using T = BsPage<D>;
  using L = BsCl<D, G>;
  const DecodeParams& p = bp.d;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);  // a value of the warp
  const int gid = lane >> 2, tig = lane & 3;
  const uint32_t ring = smem_u32(smem + warp * T::kRingBytes);
  const uint32_t bars = smem_u32(smem + L::kBarOff) + warp * T::kStages * 8;
  if (lane == 0) {
    for (int st = 0; st < T::kStages; ++st) mbar_init(bars + st * 8, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
  }
  __syncwarp();
  griddep_wait();
  griddep_launch_dependents();
  const int pair = blockIdx.x * kBsClWarps + warp;
  if (pair >= pairs) return;
  const int seq = pair / p.kv_heads, kvh = pair - seq * p.kv_heads;

  int id = 0;
  if (lane < bp.max_blocks)
    id = __ldg(p.block_tables + size_t(seq) * p.max_blocks_per_seq + lane);
  bool bad;
  const int raw = __ldg(p.context_lens + seq);
  const int cnt = flat_pages(raw, bp.max_blocks, bad);
  if (bad && kvh == 0 && lane == 0) atomicOr(&g_decode_error, kErrBadContext);
  const int len = raw < 0 ? 0 : min(raw, cnt * kBlockTokens);
  float ks = 0.f, vs = 0.f;
  if (lane < cnt) {
    if (id >= 0 && id < p.num_blocks) {
      ks = __ldg(bp.k_scales + size_t(id) * p.kv_heads + kvh);
      vs = __ldg(bp.v_scales + size_t(id) * p.kv_heads + kvh);
    } else {
      atomicOr(&g_decode_error, kErrBadBlockId);
    }
  }
  BsAcc<D, G> acc;
  const size_t row0 = size_t(seq) * p.q_heads + size_t(kvh) * G;
  bs_walk<D, G>(acc, ring, bars, tmap_k, tmap_v, p, row0, kvh, id, ks, vs, cnt, 0, 1, len, lane);
  acc.sum_l();
#pragma unroll
  for (int nh = 0; nh < BsAcc<D, G>::NH; ++nh)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int head = 8 * nh + 2 * tig + c;
      if (head >= G) continue;
      const float inv = cnt == 0 ? 0.f : 1.f / acc.l[nh][c], unit = acc.unit(nh, c);
#pragma unroll
      for (int mt = 0; mt < BsAcc<D, G>::MT; ++mt) {
        const size_t at = (row0 + head) * D + 16 * mt + 2 * gid;
        store_out(p, at, acc.value(nh, mt, c, inv, unit));
        store_out(p, at + 1, acc.value(nh, mt, c + 2, inv, unit));
      }
    }
}

// --------------------------------------------------------------- flat split
constexpr int kBsFlatMaxSeqs = 1024;
constexpr int kBsFlatWarps = 12;
// Pages of a range at least, the two that a step takes: only contexts far below the
// bound on their lengths leave warps without work (254 contexts of a token, 128 heads
// of 64 on 8: 17.0 us, 35.1 with eight pages at least; 227 of 32 / 32 of 128: 14.4, 21.7).
constexpr int kBsFlatMinPages = 2;

template <int D>
struct BsFlat {
  static constexpr int kBarOff = kBsFlatWarps * BsPage<D>::kRingBytes;
  static constexpr int kPreOff = kBarOff + kBsFlatWarps * BsPage<D>::kStages * 8;
  static constexpr int kScanOff = kPreOff + (kBsFlatMaxSeqs + 1) * 4;
  static constexpr int kSmemBytes = kScanOff + 32 * 4 + 1024;
  static_assert(kSmemBytes <= 232448, "flat decode CTA does not fit in shared memory");
};

template <int D, int G>
__global__ void __launch_bounds__(kBsFlatWarps * 32, 1)
decode_block_scaled_flat_kernel(const __grid_constant__ CUtensorMap tmap_k,
                                const __grid_constant__ CUtensorMap tmap_v,
                                const BsDecodeParams bp, const DecodeFlatParams fp) {
  using T = BsPage<D>;
  using L = BsFlat<D>;
  constexpr int kStages = T::kStages;
  constexpr int kThreads = kBsFlatWarps * 32;
  constexpr unsigned kFull = 0xffffffffu;
  const DecodeParams& p = bp.d;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int32_t* pre = reinterpret_cast<int32_t*>(smem + L::kPreOff);
  int32_t* scan = reinterpret_cast<int32_t*>(smem + L::kScanOff);
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(kFull, int(threadIdx.x >> 5), 0);  // a value of the warp
  const int gid = lane >> 2, tig = lane & 3;
  const int S = fp.num_seqs;
  const int Hkv = p.kv_heads;

  const uint32_t ring = smem_u32(smem + warp * T::kRingBytes);
  const uint32_t bars = smem_u32(smem + L::kBarOff) + warp * kStages * 8;
  if (lane == 0) {
    for (int st = 0; st < kStages; ++st) mbar_init(bars + st * 8, 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
  }
  griddep_wait();

  // ---- pages per sequence and their prefix sum, alike in every CTA
  const int per = (S + kThreads - 1) / kThreads;
  const int s_begin = threadIdx.x * per;
  int local = 0;
  for (int k = 0; k < per; ++k) {
    const int s = s_begin + k;
    if (s < S) {
      bool bad;
      const int n = flat_pages(__ldg(p.context_lens + s), fp.max_blocks, bad);
      if (bad && blockIdx.x == 0) atomicOr(&g_decode_error, kErrBadContext);
      pre[s] = n;
      local += n;
    }
  }
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int v = lane < kBsFlatWarps ? scan[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v += u;
    }
    if (lane < kBsFlatWarps) scan[lane] = v;
  }
  __syncthreads();
  {
    int base = (warp > 0 ? scan[warp - 1] : 0) + incl - local;
    for (int k = 0; k < per; ++k) {
      const int s = s_begin + k;
      if (s < S) {
        const int n = pre[s];
        pre[s] = base;
        base += n;
      }
    }
    if (threadIdx.x == 0) pre[S] = scan[kBsFlatWarps - 1];
  }
  __syncthreads();
  griddep_launch_dependents();
  if (blockIdx.x == 0)
    for (int s = threadIdx.x; s <= S; s += kThreads) fp.pre_out[s] = pre[s];

  // ---- this warp's range [f0, f1) of the blocks laid end to end, head hw
  const long long total = pre[S];
  const long long groups = flat_groups((long long)gridDim.x * kBsFlatWarps, Hkv);
  const long long gw = (long long)blockIdx.x * kBsFlatWarps + warp;
  const long long g = gw / Hkv;
  const int hw = int(gw - g * Hkv);
  const long long c = flat_chunk(total, groups, fp.min_pages);
  const long long f0 = g * c;
  const long long f1 = g >= groups ? f0 : (f0 + c < total ? f0 + c : total);
  const int cnt = f0 < f1 ? int(f1 - f0) : 0;
  if (cnt == 0) return;  // no CTA-wide barrier follows

  // Windows of 32 pages, lane k holding page 32 w + k: block id, sequence,
  // block and scales.  Copies run at most kStages pages ahead, within the
  // current window and the next; the one after is loaded a window ahead.
  struct Window {
    int id, seq, blk;
    float ks, vs;
  };
  auto load_window = [&](int win) {
    Window w = {0, -1, 0, 0.f, 0.f};
    const long long f = f0 + (long long)win * 32 + lane;
    if (f < f1) {
      int lo = 0, hi = S - 1;  // the last sequence that starts at or before f
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= f) lo = mid;
        else hi = mid - 1;
      }
      w.seq = lo;
      w.blk = int(f - pre[lo]);
      w.id = __ldg(p.block_tables + size_t(lo) * p.max_blocks_per_seq + w.blk);
      if (w.id >= 0 && w.id < p.num_blocks) {
        w.ks = __ldg(bp.k_scales + size_t(w.id) * Hkv + hw);
        w.vs = __ldg(bp.v_scales + size_t(w.id) * Hkv + hw);
      } else if (hw == 0) {
        atomicOr(&g_decode_error, kErrBadBlockId);
      }
    }
    return w;
  };
  int wcur = 0;
  Window wc = load_window(0), wn = load_window(1), wp = load_window(2);
  auto issue = [&](int j) {
    const int id = __shfl_sync(kFull, (j >> 5) == wcur ? wc.id : wn.id, j & 31);
    const int st = j % kStages;
    bs_issue<D>(ring + st * T::kStageBytes, bars + st * 8, tmap_k, tmap_v, hw, id);
  };
  for (int j = 0; j < cnt && j < kStages; ++j) issue(j);
  int issued = min(cnt, kStages);

  BsAcc<D, G> acc;
  int cur_seq = -1, cur_first = 0, cur_last = 0, cur_len = 0, cur_end = 0;
  // the finished piece: the output when it is the pair's whole context, else
  // its normalised partial, m and l at slot (sequence + g) Hkv + head (for one
  // head the pieces are ordered by sequence and range alike: no two share a slot)
  auto flush = [&]() {
    acc.sum_l();
    const bool whole = cur_first == 0 && cur_last == cur_end - 1;
    const size_t row0 = size_t(cur_seq) * p.q_heads + size_t(hw) * G;
    const size_t slot = (size_t(cur_seq) + size_t(g)) * Hkv + hw;
#pragma unroll
    for (int nh = 0; nh < BsAcc<D, G>::NH; ++nh)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const int head = 8 * nh + 2 * tig + cc;
        if (head >= G) continue;
        const float inv = 1.f / acc.l[nh][cc], unit = acc.unit(nh, cc);
#pragma unroll
        for (int mt = 0; mt < BsAcc<D, G>::MT; ++mt) {
          const int dim = 16 * mt + 2 * gid;
          const float v0 = acc.value(nh, mt, cc, inv, unit),
                      v1 = acc.value(nh, mt, cc + 2, inv, unit);
          if (whole) {
            store_out(p, (row0 + head) * D + dim, v0);
            store_out(p, (row0 + head) * D + dim + 1, v1);
          } else {
            *reinterpret_cast<float2*>(p.part_o + (slot * G + head) * D + dim) = make_float2(v0, v1);
          }
        }
        if (!whole && gid == 0)
          bp.part_ml[slot * G + head] = make_float2(acc.m[nh][cc], acc.l[nh][cc]);
      }
  };

  bool failed = false;
  int i = 0;
  while (i < cnt) {
    const bool in0 = (i >> 5) == wcur, in1 = ((i + 1) >> 5) == wcur;
    const int seq0 = __shfl_sync(kFull, in0 ? wc.seq : wn.seq, i & 31);
    const int blk0 = __shfl_sync(kFull, in0 ? wc.blk : wn.blk, i & 31);
    const int seq1 = __shfl_sync(kFull, in1 ? wc.seq : wn.seq, (i + 1) & 31);
    const bool two = i + 1 < cnt && seq1 == seq0;
    if (seq0 != cur_seq) {
      if (cur_seq >= 0) flush();
      cur_seq = seq0;
      cur_first = blk0;
      cur_end = pre[seq0 + 1] - pre[seq0];
      const int raw = __ldg(p.context_lens + seq0);
      cur_len = raw < cur_end * kBlockTokens ? raw : cur_end * kBlockTokens;
      acc.start(p.q, size_t(seq0) * p.q_heads + size_t(hw) * G, p.scale_log2, lane);
    }
    bool landed = mbar_wait_bounded(bars + (i % kStages) * 8, (i / kStages) & 1);
    if (two && landed)
      landed = mbar_wait_bounded(bars + ((i + 1) % kStages) * 8, ((i + 1) / kStages) & 1);
    if (!__all_sync(kFull, landed)) {
      failed = true;
      break;
    }
    const uint32_t b0 = ring + (i % kStages) * T::kStageBytes;
    const float ks0 = __shfl_sync(kFull, in0 ? wc.ks : wn.ks, i & 31);
    const float vs0 = __shfl_sync(kFull, in0 ? wc.vs : wn.vs, i & 31);
    if (two) {
      const uint32_t kb[2] = {b0, ring + ((i + 1) % kStages) * T::kStageBytes};
      const int tk[2] = {blk0 * kBlockTokens, (blk0 + 1) * kBlockTokens};
      const float k2[2] = {ks0, __shfl_sync(kFull, in1 ? wc.ks : wn.ks, (i + 1) & 31)};
      const float v2[2] = {vs0, __shfl_sync(kFull, in1 ? wc.vs : wn.vs, (i + 1) & 31)};
      bs_pages<D, G, 2>(acc, kb, tk, k2, v2, cur_len, lane);
    } else {
      const uint32_t kb[1] = {b0};
      const int tk[1] = {blk0 * kBlockTokens};
      const float k1[1] = {ks0}, v1[1] = {vs0};
      bs_pages<D, G, 1>(acc, kb, tk, k1, v1, cur_len, lane);
    }
    cur_last = blk0 + (two ? 1 : 0);
    __syncwarp();
    const int n = two ? 2 : 1;
    for (int j = i; j < i + n; ++j)
      if (j + kStages < cnt) {
        issue(j + kStages);
        ++issued;
      }
    i += n;
    if ((i >> 5) != wcur && i < cnt) {
      wcur = i >> 5;
      wc = wn;
      wn = wp;
      wp = load_window(wcur + 2);
    }
  }
  if (failed) {
    if (lane == 0) {
      atomicOr(&g_decode_error, kErrWaitTimeout);
      for (int k = i; k < issued; ++k)
        (void)mbar_wait_bounded(bars + (k % kStages) * 8, (k / kStages) & 1);
    }
    __syncwarp();
    return;
  }
  flush();
}

// Joins the pieces of a cut pair: row (sequence s, query head) of KV head h;
// the pages [pre[s], pre[s] + n) lie in the ranges g0 = pre[s] / c .. g1 =
// (pre[s] + n - 1) / c, range g's piece at slot (s + g) Hkv + h.  An empty
// sequence gets zeros; a pair within one range is written already.  WPR warps
// take a row's pieces, 16 (4) at a time each, with all their loads in flight at
// once -- lane i reads piece i's maximum and sum -- and join their sums in shared
// memory: with few rows each has a hundred pieces, and it is round trips that
// count (2 x 131072 tokens, 114 pieces: 39 us for one warp and eight loads in
// flight, 5.0 now); with many rows there are two or none.
template <int D, int WPR>
__global__ void __launch_bounds__(256)
decode_block_scaled_merge_kernel(const BsDecodeParams bp, const DecodeFlatParams fp,
                                 long long total_rows) {
  const DecodeParams& p = bp.d;
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kCols = D / 32;  // a lane's elements
  constexpr int kBatch = WPR > 1 ? 16 : 4;
  constexpr unsigned kFull = 0xffffffffu;
  __shared__ float part[WPR > 1 ? WPR : 1][WPR > 1 ? D + 2 : 1];  // O, then maximum and sum
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = warp % WPR;
  const long long row = (long long)blockIdx.x * (8 / WPR) + warp / WPR;
  if (row >= total_rows) return;  // WPR 8: the whole CTA
  const int seq = int(row / p.q_heads);
  const int hq = int(row - (long long)seq * p.q_heads);
  const int G = p.q_heads / p.kv_heads;
  const int h = hq / G, hg = hq - h * G;
  const int start = __ldg(fp.pre_out + seq), n = __ldg(fp.pre_out + seq + 1) - start;
  const long long c = flat_chunk(__ldg(fp.pre_out + fp.num_seqs),
                                 flat_groups(fp.total_warps, p.kv_heads), fp.min_pages);
  const int g0 = int(start / c), g1 = n > 0 ? int((start + n - 1) / c) : g0 - 1;
  if (g1 == g0) return;
  auto slot = [&](int g) { return (size_t(seq + g) * p.kv_heads + h) * G + hg; };
  float big = -INFINITY, tot = 0.f, val[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) val[i] = 0.f;
  for (int b = g0 + w * kBatch; b <= g1; b += WPR * kBatch) {
    const int cnt = min(kBatch, g1 - b + 1);
    const float2 ml =
        lane < cnt ? __ldg(bp.part_ml + slot(b + lane)) : make_float2(-INFINITY, 0.f);
    float x[kBatch][kCols];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float* src = p.part_o + slot(b + min(i, cnt - 1)) * D + lane * kCols;
      if constexpr (kCols == 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(src));
        x[i][0] = v.x;
        x[i][1] = v.y;
        x[i][2] = v.z;
        x[i][3] = v.w;
      } else {
        const float2 v = __ldg(reinterpret_cast<const float2*>(src));
        x[i][0] = v.x;
        x[i][1] = v.y;
      }
    }
    float top = ml.x;
#pragma unroll
    for (int o = kBatch / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    top = fmaxf(big, __shfl_sync(kFull, top, 0));
    const float alpha = big == top ? 1.f : ex2(big - top);  // (-inf: 0, or nothing yet)
    big = top;
    const float mine = lane < cnt ? ml.y * ex2(ml.x - top) : 0.f;
    float sum = mine;
#pragma unroll
    for (int o = kBatch / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    tot = tot * alpha + __shfl_sync(kFull, sum, 0);
#pragma unroll
    for (int k = 0; k < kCols; ++k) val[k] *= alpha;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float f = __shfl_sync(kFull, mine, i);
      if (i < cnt)
#pragma unroll
        for (int k = 0; k < kCols; ++k) val[k] += f * x[i][k];
    }
  }
  if constexpr (WPR == 1) {
    const float inv = n > 0 ? 1.f / tot : 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) store_out(p, size_t(row) * D + lane * kCols + i, val[i] * inv);
  } else {
#pragma unroll
    for (int i = 0; i < kCols; ++i) part[w][lane * kCols + i] = val[i];
    if (lane == 0) {
      part[w][D] = big;
      part[w][D + 1] = tot;
    }
    __syncthreads();
    for (int x = threadIdx.x; x < D; x += 256) {
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < WPR; ++k) top = fmaxf(top, part[k][D]);
      float sum = 0.f, all = 0.f;
#pragma unroll
      for (int k = 0; k < WPR; ++k) {
        // a warp without pieces has a sum of 0 and no maximum
        const float f = part[k][D + 1] == 0.f ? 0.f : ex2(part[k][D] - top);
        sum += f * part[k][x];
        all += f * part[k][D + 1];
      }
      store_out(p, size_t(row) * D + x, n > 0 ? sum / all : 0.f);
    }
  }
}

// ------------------------------------------------------------------- launch
namespace {

template <int D>
cudaError_t launch_merge(const BsDecodeParams& bp, const DecodeFlatParams& fp, int ctas,
                         cudaStream_t stream) {
  const long long rows = (long long)fp.num_seqs * bp.d.q_heads;
  const bool few = rows <= 8ll * ctas;
  const long long grid = few ? rows : (rows + 7) / 8;
  if (grid > INT_MAX) return cudaErrorInvalidValue;
  return few ? launch_after_previous(decode_block_scaled_merge_kernel<D, 8>,
                                     dim3(unsigned(grid)), dim3(256), 0, stream, bp, fp, rows)
             : launch_after_previous(decode_block_scaled_merge_kernel<D, 1>,
                                     dim3(unsigned(grid)), dim3(256), 0, stream, bp, fp, rows);
}

template <int D, int G>
cudaError_t launch_cluster(const BsDecodeParams& bp, int num_seqs, int ctas,
                           const CUtensorMap* tk, const CUtensorMap* tv, cudaStream_t stream) {
  using L = BsCl<D, G>;
  static std::atomic<int> attr_done[kAttrMaxDevices];
  cudaError_t e = set_smem_limit_once(decode_block_scaled_cluster_kernel<D, G>, L::kSmemBytes,
                                      attr_done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(num_seqs * bp.d.kv_heads * ctas));
  cfg.blockDim = dim3(kBsClWarps * 32);
  cfg.dynamicSmemBytes = L::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(ctas);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, decode_block_scaled_cluster_kernel<D, G>, *tk, *tv, bp);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int D, int G>
cudaError_t launch_pairs(const BsDecodeParams& bp, int num_seqs, const CUtensorMap* tk,
                         const CUtensorMap* tv, cudaStream_t stream) {
  constexpr int kSmem = BsCl<D, G>::kOutOff + 1024;  // rings and barriers
  static std::atomic<int> attr_done[kAttrMaxDevices];
  cudaError_t e = set_smem_limit_once(decode_block_scaled_pairs_kernel<D, G>, kSmem, attr_done);
  if (e != cudaSuccess) return e;
  const int pairs = num_seqs * bp.d.kv_heads;
  return launch_after_previous(decode_block_scaled_pairs_kernel<D, G>,
                               dim3(unsigned((pairs + kBsClWarps - 1) / kBsClWarps)),
                               dim3(kBsClWarps * 32), kSmem, stream, *tk, *tv, bp, pairs);
}

template <int D, int G>
cudaError_t launch_flat(const BsDecodeParams& bp, const DecodeFlatParams& fp, int ctas,
                        const CUtensorMap* tk, const CUtensorMap* tv, cudaStream_t stream) {
  using L = BsFlat<D>;
  static std::atomic<int> attr_done[kAttrMaxDevices];
  cudaError_t e =
      set_smem_limit_once(decode_block_scaled_flat_kernel<D, G>, L::kSmemBytes, attr_done);
  if (e != cudaSuccess) return e;
  e = launch_after_previous(decode_block_scaled_flat_kernel<D, G>, dim3(unsigned(ctas)),
                            dim3(kBsFlatWarps * 32), L::kSmemBytes, stream, *tk, *tv, bp, fp);
  if (e != cudaSuccess) return e;
  return launch_merge<D>(bp, fp, ctas, stream);
}

// CTAs of a pair's cluster, or 0 for the flat split.
int cluster_ctas(long long pairs, int max_blocks, int num_sms) {
  const long long slots = 3ll * num_sms;
  int c = 1;
  while (c < kBsClMaxCtas && pairs * c * 2 <= slots && max_blocks > 2 * c * kBsClWarps) c *= 2;
  if (pairs * c > slots || max_blocks > c * kBsClWarps * kBsClMaxPages) return 0;
  return c;
}

}  // namespace

int decode_block_scaled_warps() { return kBsFlatWarps; }
int decode_block_scaled_flat_seqs() { return kBsFlatMaxSeqs; }

cudaError_t launch_decode_block_scaled(const DecodeBlockScaledArgs& a, const CUtensorMap* tk,
                                       const CUtensorMap* tv, int num_sms, cudaStream_t stream) {
  const int group = a.q_heads / a.kv_heads;
  const size_t elem = a.out_bf16 ? 2 : 4;
  const int max_blocks = std::min(a.max_blocks_per_seq, (a.max_context_len - 1) / kBlockTokens + 1);
  BsDecodeParams bp = {};
  DecodeParams& d = bp.d;
  d.part_o = a.part_o;
  d.q_heads = a.q_heads;
  d.kv_heads = a.kv_heads;
  d.num_blocks = a.num_blocks;
  d.max_blocks_per_seq = a.max_blocks_per_seq;
  d.scale_log2 = a.scale_log2;
  d.out_scale = 1.f;
  d.out_bf16 = a.out_bf16 ? 1 : 0;
  bp.k_scales = a.k_scales;
  bp.v_scales = a.v_scales;
  bp.part_ml = a.part_ml;
  bp.max_blocks = max_blocks;
  const long long all_pairs = (long long)a.num_seqs * a.kv_heads;
  const int ctas = cluster_ctas(all_pairs, max_blocks, num_sms);
  // the flat split's prefix sums hold 1024 sequences, and 2^31 pages: more go in turn
  const bool alone = ctas == 0 && max_blocks <= kBsClMaxPages;
  const int chunk = ctas || alone ? a.num_seqs : std::min(kBsFlatMaxSeqs, INT_MAX / max_blocks);
  for (int s = 0; s < a.num_seqs; s += chunk) {
    const int n = std::min(chunk, a.num_seqs - s);
    const size_t row = size_t(s) * a.q_heads * a.d_head;
    d.q = static_cast<const __nv_bfloat16*>(a.q) + row;
    d.out = reinterpret_cast<float*>(static_cast<char*>(a.out) + row * elem);
    d.block_tables = a.block_tables + size_t(s) * a.max_blocks_per_seq;
    d.context_lens = a.context_lens + s;
    DecodeFlatParams fp;
    fp.pre_out = a.pre;
    fp.num_seqs = n;
    fp.max_blocks = max_blocks;
    fp.total_warps = num_sms * kBsFlatWarps;
    fp.min_pages = kBsFlatMinPages;
    cudaError_t e = cudaErrorInvalidValue;
#define PKV_BS_CASE(DD, GG)                                                       \
  if (a.d_head == DD && group == GG)                                              \
    e = ctas    ? launch_cluster<DD, GG>(bp, n, ctas, tk, tv, stream)             \
        : alone ? launch_pairs<DD, GG>(bp, n, tk, tv, stream)                     \
                : launch_flat<DD, GG>(bp, fp, num_sms, tk, tv, stream)
    PKV_BS_CASE(128, 1);
    PKV_BS_CASE(128, 2);
    PKV_BS_CASE(128, 4);
    PKV_BS_CASE(128, 8);
    PKV_BS_CASE(128, 16);
    PKV_BS_CASE(64, 1);
    PKV_BS_CASE(64, 2);
    PKV_BS_CASE(64, 4);
    PKV_BS_CASE(64, 8);
    PKV_BS_CASE(64, 16);
#undef PKV_BS_CASE
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Device address of this unit's error word on the current device.
cudaError_t decode_block_scaled_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_decode_error);
}

unsigned read_decode_block_scaled_error(bool clear) {
  unsigned word = 0;
  if (cudaMemcpyFromSymbol(&word, g_decode_error, sizeof(word)) != cudaSuccess) return ~0u;
  if (clear) {
    const unsigned zero = 0;
    if (cudaMemcpyToSymbol(g_decode_error, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  }
  return word;
}

}  // namespace pkv
