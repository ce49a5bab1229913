// The block-scaled FP8 cache: pools of e4m3 codes with one float32 scale for
// each block of 16 tokens and KV head, [num_blocks][kv_heads].  Here: the
// quantizing append, the widening of pages to bf16 rows for the prefill, and
// the copy of scales that goes with a block copy.  (The decode is
// paged_decode_block_scaled.cu.)
//
// The append.  For a block b and KV head h let x be the new rows that the call
// writes into b.  Its scale becomes
//   s = max(s_old, 2^e),  e = min{ e >= -126 : max |x| <= 448 2^e },
// s_old counting only if older rows of the sequence lie before x in b; new
// rows are stored as e4m3(x / s), older ones as e4m3(code s_old / s) when s
// grew.  Powers of two: dividing by one rounds nothing, so a code is the
// element rounded once; an older code moved to a larger scale only changes
// where it falls among e4m3's subnormals; and a wider format holds code times
// scale exactly (below 2^128).  A scale from the largest value itself would use up to one
// bit more of e4m3's range, but none of its three fraction bits.
//
// One warp takes one (block, KV head, K or V): its up to 16 rows are in
// registers between the maximum and the stores, so the inputs are read once.
// Bound by HBM for prompts (8 chunks of 1025 to 2048 tokens, 8 heads of 128: 15.1
// us with inputs that are not in L2, 0.68 of the copy rate; the same inputs again and
// again 12.3, and 15.1 with finite elements picked one by one and three CTAs an SM),
// by launch and three round trips for single tokens.
// Which rows form a block follows from q_start and the context lengths.
#include <algorithm>
#include <climits>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tcgen05.cuh"  // packed float32 arithmetic

namespace pkv {

static __device__ unsigned g_block_scaled_error = 0;

constexpr int kBsTokens = 16;     // tokens per block
constexpr int kBsThreads = 256;
constexpr int kBsMaxRows = 16;    // new rows per CTA at most
constexpr int kSplitPerSm = 3;    // CTAs per SM up to which a block's tasks are spread

// The scale of values up to `amax` (bf16 bits of the largest finite
// magnitude): 1.75 is 448's fraction, so a larger fraction needs one more.
__device__ __forceinline__ float block_scale(uint32_t amax_bf16) {
  const int e = int(((amax_bf16 << 16) + 0x1fffffu) >> 23) - 135;
  return __uint_as_float(uint32_t(max(e, -126) + 127) << 23);
}

// The larger magnitudes of two bf16 pairs; FINITE: infinities and NaN left out.
template <bool FINITE>
__device__ __forceinline__ uint32_t magnitude_max2(uint32_t m, uint32_t w) {
  const uint32_t a = w & 0x7fff7fffu;
  return __vmaxu2(m, FINITE ? a & __vcmpltu2(a, 0x7f807f80u) : a);
}
template <bool FINITE, int N>
__device__ __forceinline__ uint32_t largest(const uint4 (&x)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m = magnitude_max2<FINITE>(m, x[i].x);
    m = magnitude_max2<FINITE>(m, x[i].y);
    m = magnitude_max2<FINITE>(m, x[i].z);
    m = magnitude_max2<FINITE>(m, x[i].w);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  return max(m & 0xffffu, m >> 16);
}

// Four floats -> four e4m3 codes (nearest even, finite overflow to +-448).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Two bf16 pairs times a factor -> four e4m3 codes.
__device__ __forceinline__ uint32_t quantized(uint32_t a, uint32_t b, uint64_t factor2) {
  float f[4];
  f2_unpack(f2_mul(f2_pack(bf16_lo_to_f32(a), bf16_hi_to_f32(a)), factor2), f[0], f[1]);
  f2_unpack(f2_mul(f2_pack(bf16_lo_to_f32(b), bf16_hi_to_f32(b)), factor2), f[2], f[3]);
  return e4m3x4(f[0], f[1], f[2], f[3]);
}

// Four e4m3 codes -> floats (exact, through f16).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t codes, float (&f)[4]) {
  asm("{\n\t.reg .b16 c0, c1, h0, h1, h2, h3;\n\t.reg .b32 a, b;\n\t"
      "mov.b32 {c0, c1}, %4;\n\t"
      "cvt.rn.f16x2.e4m3x2 a, c0;\n\t"
      "cvt.rn.f16x2.e4m3x2 b, c1;\n\t"
      "mov.b32 {h0, h1}, a;\n\t"
      "mov.b32 {h2, h3}, b;\n\t"
      "cvt.f32.f16 %0, h0;\n\t"
      "cvt.f32.f16 %1, h1;\n\t"
      "cvt.f32.f16 %2, h2;\n\t"
      "cvt.f32.f16 %3, h3;\n\t}"
      : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
      : "r"(codes));
}

__device__ __forceinline__ uint32_t rescaled(uint32_t codes, float ratio) {
  float f[4];
  e4m3x4_to_f32(codes, f);
  return e4m3x4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
}

// One (block, head) of one tensor, by one warp: `count` new rows from `src`
// (stride elements apart) to the block's rows [first, first + count).
template <int D>
__device__ __forceinline__ void append_block(const __nv_bfloat16* __restrict__ src, int64_t stride,
                                             uint8_t* __restrict__ block, int row_bytes,
                                             float* __restrict__ scale, int first, int count) {
  constexpr int kLanes = D / 8;           // lanes of a row, 8 elements each
  constexpr int kRows = 32 / kLanes;      // rows of a step
  constexpr int kSteps = kBsTokens / kRows;
  const int lane = threadIdx.x & 31;
  const int sub = lane / kLanes, col = (lane % kLanes) * 8;
  const float old = first > 0 ? __ldcg(scale) : 0.f;
  uint4 x[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = i * kRows + sub;
    x[i] = r < count ? __ldg(reinterpret_cast<const uint4*>(src + r * stride + col))
                     : make_uint4(0, 0, 0, 0);
  }
  uint32_t top = largest<false>(x);
  if (top >= 0x7f80u) top = largest<true>(x);  // an infinity or NaN among them
  const float s = fmaxf(old, block_scale(top));
  const float inv = 1.f / s;  // exact for a power of two
  const uint64_t inv2 = f2_pack(inv, inv);
  uint8_t* dst = block + size_t(first) * row_bytes + col;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = i * kRows + sub;
    if (r < count) {
      const uint4 w = x[i];
      *reinterpret_cast<uint2*>(dst + size_t(r) * row_bytes) =
          make_uint2(quantized(w.x, w.y, inv2), quantized(w.z, w.w, inv2));
    }
  }
  if (s != old) {
    if (first > 0) {  // the older rows move to the larger scale
      const float ratio = old * inv;
      for (int r = sub; r < first; r += kRows) {
        uint2* at = reinterpret_cast<uint2*>(block + size_t(r) * row_bytes + col);
        const uint2 w = *at;
        *at = make_uint2(rescaled(w.x, ratio), rescaled(w.y, ratio));
      }
    }
    if (lane == 0) *scale = s;
  }
}

// CTA (x, y): the blocks whose first new rows are among rows [x rows_per_cta,
// ...), the y-th part of their (head, K or V) tasks.
template <int D>
__global__ void __launch_bounds__(kBsThreads, 4)
append_block_scaled_kernel(const AppendBlockScaledArgs a, int rows_per_cta) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int items, fall, item_row[kBsMaxRows], item_first[kBsMaxRows],
      item_count[kBsMaxRows], item_block[kBsMaxRows];
  if (threadIdx.x == 0) {
    items = 0;
    fall = a.num_seqs;
  }
  __syncthreads();
  // every sequence looks for its blocks that start among these rows
  const int64_t r0 = int64_t(blockIdx.x) * rows_per_cta;
  const int64_t r1 = min(r0 + rows_per_cta, a.total);
  const bool first_cta = blockIdx.x == 0 && blockIdx.y == 0;
  auto find = [&](int seqs) {
    bool falls = false;
    for (int s = threadIdx.x; s < seqs; s += kBsThreads) {
      const int qs = __ldg(a.q_start + s), qe = __ldg(a.q_start + s + 1);
      const int ctx = __ldg(a.context_lens + s);
      const int n = qe - qs;
      if (qs < 0 || qe < qs || qe > a.total || n > ctx || ctx > a.max_blocks_per_seq * kBsTokens) {
        if (n != 0 && first_cta) atomicOr(&g_block_scaled_error, kErrBadQueryRange);
        if (qe < qs) {
          falls = true;
          atomicMin(&fall, s);
        }
        continue;
      }
      const int base = ctx - n - qs;  // position of row r: base + r
      const int64_t hi = min(int64_t(qe), r1);
      int64_t r = max(int64_t(qs), r0);
      if (r > qs) r += (kBsTokens - (base + r) % kBsTokens) % kBsTokens;  // the next block's start
      while (r < hi) {
        const int pos = int(base + r), first = pos % kBsTokens;
        const int block = __ldg(a.block_tables + size_t(s) * a.max_blocks_per_seq + pos / kBsTokens);
        const int rows = min(kBsTokens - first, int(qe - r));
        if (block < 0 || block >= a.num_blocks) {
          atomicOr(&g_block_scaled_error, kErrBadBlockId);
        } else {
          const int at = atomicAdd(&items, 1);
          if (at < kBsMaxRows) {  // (more only where sequences claim the same rows)
            item_row[at] = int(r - r0);
            item_first[at] = first;
            item_count[at] = rows;
            item_block[at] = block;
          }
        }
        r += rows;
      }
    }
    return falls;
  };
  // Where starts fall, the sequence that ends before it begins and all behind it are
  // left out: the others lie behind one another, a block's first row each.
  if (__syncthreads_or(find(a.num_seqs))) {
    if (threadIdx.x == 0) items = 0;
    __syncthreads();
    find(fall);
    __syncthreads();
  }
  const int row_bytes = a.kv_heads * D;
  const int tasks = items * a.kv_heads * 2;
  for (int t = int(blockIdx.y) * (kBsThreads / 32) + (threadIdx.x >> 5); t < tasks;
       t += gridDim.y * (kBsThreads / 32)) {
    const int item = t / (2 * a.kv_heads), rest = t - item * 2 * a.kv_heads;
    const bool v = rest >= a.kv_heads;
    const int h = v ? rest - a.kv_heads : rest;
    const int64_t r = r0 + item_row[item];
    const int block = item_block[item];
    const int64_t stride = v ? a.v_stride : a.k_stride;
    append_block<D>((v ? a.v : a.k) + r * stride + h * D, stride,
                    (v ? a.v_cache : a.k_cache) + size_t(block) * kBsTokens * row_bytes + h * D,
                    row_bytes, (v ? a.v_scales : a.k_scales) + size_t(block) * a.kv_heads + h,
                    item_first[item], item_count[item]);
  }
}

cudaError_t launch_append_block_scaled(const AppendBlockScaledArgs& a, int d_head, int num_sms,
                                       cudaStream_t stream) {
  // About one block's first row per CTA: a batch of single tokens gives every
  // token a CTA, a prompt every block.  Few of them: a block's tasks are
  // spread over several CTAs, down to one for each warp (one token of 32
  // heads: 10.9 us with all tasks in one CTA, 2.7 so).
  const int64_t firsts = std::min(a.total, a.total / kBsTokens + a.num_seqs);
  int rows = 1;
  while (rows < kBsMaxRows && int64_t(rows) * 2 * firsts <= a.total) rows *= 2;
  const int64_t grid = (a.total + rows - 1) / rows;
  if (grid > INT_MAX) return cudaErrorInvalidValue;
  const int parts = (2 * a.kv_heads + kBsThreads / 32 - 1) / (kBsThreads / 32);
  int split = 1;
  while (split < parts && split < 1024 && grid * split < kSplitPerSm * int64_t(num_sms)) split *= 2;
  auto* kernel = d_head == 128 ? append_block_scaled_kernel<128> : append_block_scaled_kernel<64>;
  return launch_after_previous(kernel, dim3(unsigned(grid), unsigned(split)), dim3(kBsThreads), 0,
                               stream, a, rows);
}

// The scales' part of a block copy: row dst of both arrays becomes row src.
__global__ void __launch_bounds__(128)
copy_block_scales_kernel(float* __restrict__ k_scales, float* __restrict__ v_scales,
                         const int32_t* __restrict__ pairs, int num_pairs, int num_blocks,
                         int kv_heads) {
  const int64_t all = 2ll * num_pairs * kv_heads;
  for (int64_t i = int64_t(blockIdx.x) * 128 + threadIdx.x; i < all; i += int64_t(gridDim.x) * 128) {
    const int64_t p = i / (2 * kv_heads);
    const int c = int(i - p * 2 * kv_heads);
    const int32_t src = __ldg(pairs + 2 * p), dst = __ldg(pairs + 2 * p + 1);
    if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) {
      if (c == 0) atomicOr(&g_block_scaled_error, kErrBadBlockId);
      continue;
    }
    float* x = c < kv_heads ? k_scales + c : v_scales + (c - kv_heads);
    x[size_t(dst) * kv_heads] = x[size_t(src) * kv_heads];
  }
}

cudaError_t launch_copy_block_scales(float* k_scales, float* v_scales, const int32_t* pairs,
                                     int num_pairs, int num_blocks, int kv_heads,
                                     cudaStream_t stream, int num_sms) {
  const int64_t want = (2ll * num_pairs * kv_heads + 127) / 128;
  const int grid = int(std::min<int64_t>(want, int64_t(num_sms) * 8));
  copy_block_scales_kernel<<<grid, 128, 0, stream>>>(k_scales, v_scales, pairs, num_pairs,
                                                     num_blocks, kv_heads);
  return cudaGetLastError();
}

// Pages -> contiguous bf16 rows for the prefill: position t of sequence s to row
// s * max_blocks * 16 + t of both outputs.  code * scale is a bf16 value for the
// append's scales; other scales' products are rounded to one.  Bound by HBM (one
// byte read, two written an element).  A CTA takes a page of K and V, a thread
// four times 16 codes at once, which lie in one head each; the next page's
// number is on its way meanwhile.  Pages of sequences without new rows are nobody's.
__global__ void __launch_bounds__(kBsThreads)
widen_block_scaled_kernel(const WidenBlockScaledArgs a, int d_head) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t items = int64_t(a.num_seqs) * a.max_blocks_per_seq;
  const int row_vec = a.kv_heads * d_head / 16;  // 16 codes each
  const int page_vec = kBsTokens * row_vec;
  const int head_vec = d_head / 16;
  // the page's number and its rows in use; none: 0 rows
  auto page_of = [&](int64_t item, int& id, int& live) {
    live = 0;
    if (item >= items) return;
    const int s = int(item / a.max_blocks_per_seq);
    const int new_rows = __ldg(a.q_start + s + 1) - __ldg(a.q_start + s);
    live = __ldg(a.context_lens + s) - int(item - int64_t(s) * a.max_blocks_per_seq) * kBsTokens;
    if (new_rows <= 0) live = 0;
    if (live > 0) id = __ldg(a.block_tables + item);
  };
  int id = 0, live;
  page_of(blockIdx.x, id, live);
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    int next_id = 0, next_live;
    page_of(item + gridDim.x, next_id, next_live);
    if (live > 0) {
      const bool good = id >= 0 && id < a.num_blocks;
      if (!good && threadIdx.x == 0) atomicOr(&g_block_scaled_error, kErrBadBlockId);
      const int used = min(live, kBsTokens) * row_vec;  // of page_vec
      constexpr int kBatch = 4;
#pragma unroll 1
      for (int i0 = threadIdx.x; i0 < 2 * used; i0 += kBatch * kBsThreads) {
        uint4 w[kBatch];
        float f[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int i = i0 + u * kBsThreads;
          const bool v = i >= used;
          const int c = v ? i - used : i;
          w[u] = make_uint4(0, 0, 0, 0);
          f[u] = 0.f;
          if (good && i < 2 * used) {
            w[u] = __ldg(reinterpret_cast<const uint4*>(v ? a.v_cache : a.k_cache) +
                         size_t(id) * page_vec + c);
            f[u] = __ldg((v ? a.v_scales : a.k_scales) + size_t(id) * a.kv_heads +
                         c % row_vec / head_vec);
          }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int i = i0 + u * kBsThreads;
          if (i >= 2 * used) break;
          const bool v = i >= used;
          const int c = v ? i - used : i;
          const uint32_t in[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
          uint32_t out[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float x[4];
            e4m3x4_to_f32(in[k], x);
            out[2 * k] = pack_bf16x2(x[0] * f[u], x[1] * f[u]);
            out[2 * k + 1] = pack_bf16x2(x[2] * f[u], x[3] * f[u]);
          }
          char* dst = static_cast<char*>(v ? a.v_out : a.k_out) + (item * page_vec + c) * 32;
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst),
                       "r"(out[0]), "r"(out[1]), "r"(out[2]), "r"(out[3]), "r"(out[4]),
                       "r"(out[5]), "r"(out[6]), "r"(out[7])
                       : "memory");
        }
      }
    }
    id = next_id;
    live = next_live;
  }
}

cudaError_t launch_widen_block_scaled(const WidenBlockScaledArgs& a, int d_head, int num_sms,
                                      cudaStream_t stream) {
  const int64_t items = int64_t(a.num_seqs) * a.max_blocks_per_seq;
  const int grid = int(std::min<int64_t>(items, int64_t(num_sms) * 6));
  return launch_after_previous(widen_block_scaled_kernel, dim3(unsigned(grid)), dim3(kBsThreads),
                               0, stream, a, d_head);
}

// Device address of this unit's error word on the current device.
cudaError_t block_scaled_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_block_scaled_error);
}

unsigned read_block_scaled_error(bool clear) {
  unsigned word = 0;
  if (cudaMemcpyFromSymbol(&word, g_block_scaled_error, sizeof(word)) != cudaSuccess) return ~0u;
  if (clear) {
    const unsigned zero = 0;
    if (cudaMemcpyToSymbol(g_block_scaled_error, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  }
  return word;
}

}  // namespace pkv
