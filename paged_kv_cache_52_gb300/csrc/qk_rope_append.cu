// Per-head RMS norm and rotary position embedding of new queries and keys,
// fused with the append of keys and values into the paged pools.
//
// Mathematics, for a head x of d elements (a query or a key head of a token
// at position p, weights w):
//   y = x * rsqrt(mean(x^2) + eps) * w            (without w: y = x)
//   pairs (a, b) of the first rot elements turn by the angle whose cosine c
//   and sine s are table[p][i], table[p][rot/2 + i]:
//     a' = a c - b s,  b' = b c + a s
//   with pair i = (i, i + rot/2), or (2i, 2i + 1) when interleaved; elements
//   from rot on pass through.
// Everything is float32 from the bf16 inputs on; q', k' are rounded once, to
// bf16 or (keys and values of FP8 pools) to e4m3.
//
// Bound by memory: each q, k, v element is read once and written once; what
// has to be kept low beside that are the instructions per element.  A lane
// holds two runs of 4 elements that are each other's partners (i, i + rot/2),
// so a pair never leaves its lane; d / 8 lanes make a head, and a norm is
// log2(d / 8) shuffles.  A warp takes kRows x (256 / d) heads of one token and
// one kind (q, k or v): the products of the weights with the cosines and
// sines are made once for all of them, and a rotation is then two packed
// multiply-adds for two elements.
#include <cuda_fp8.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tcgen05.cuh"

namespace pkv {

static __device__ unsigned g_rope_error = 0;

constexpr int kRopeThreads = 128;

// Two packed bf16 as two packed floats.
__device__ __forceinline__ uint64_t f2_of_bf16x2(uint32_t v) {
  return f2_pack(bf16_lo_to_f32(v), bf16_hi_to_f32(v));
}

__device__ __forceinline__ uint32_t bf16x2_of_f2(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return pack_bf16x2(a, b);
}

__device__ __forceinline__ uint32_t e4m3x4_of_f2(uint64_t v, uint64_t w) {
  float a, b, c, d;
  f2_unpack(v, a, b);
  f2_unpack(w, c, d);
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return (lo & 0xffffu) | (hi << 16);
}

// ROWS: heads in flight per lane.  Nine CTAs an SM (56 registers) measured best
// with ROWS 4: 16384 tokens into FP8 pools 104.5 us (6.2 TB/s, 0.91 of the
// measured copy rate), 109 with 8 CTAs, 108 with 10, 110 with 12.
template <int D, bool INTERLEAVED, bool FP8, int ROWS>
__global__ void __launch_bounds__(kRopeThreads, 9)
qk_rope_append_kernel(const QkRopeArgs p) {
  griddep_wait();  // inputs may have been written by the previous kernel in the stream
  constexpr int LPH = D / 8;       // lanes per head
  constexpr int HPR = 32 / LPH;    // heads a warp holds side by side
  constexpr int HPU = ROWS * HPR;  // heads per warp
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t(blockIdx.x) * kRopeThreads + threadIdx.x) >> 5;
  const int q_units = (p.q_heads + HPU - 1) / HPU, kv_units = (p.kv_heads + HPU - 1) / HPU;
  const int units = q_units + 2 * kv_units;  // warps per token
  const int64_t t = unit / units;
  if (t >= p.num_tokens) return;
  const int u = int(unit - t * units);
  const bool is_q = u < q_units, is_v = u >= q_units + kv_units;
  const int h0 = (is_q ? u : (is_v ? u - q_units - kv_units : u - q_units)) * HPU + lane / LPH;
  const int heads = is_q ? p.q_heads : p.kv_heads;
  const int hl = lane % LPH;
  // this lane's two runs of 4 elements: partners, or (interleaved, and beyond
  // the rotated elements) neighbours
  const bool turns = 8 * hl < p.rot_dim;
  const bool apart = !INTERLEAVED && turns;
  const int ea = apart ? 4 * hl : 8 * hl;
  const int eb = apart ? ea + p.rot_dim / 2 : ea + 4;

  const int64_t pos = __ldg(p.positions + t);
  const int64_t slot = __ldg(p.slot_mapping + t);
  const __nv_bfloat16* src = is_q ? p.q + t * p.q_stride : (is_v ? p.v + t * p.v_stride
                                                                 : p.k + t * p.k_stride);
  uint2 xa[ROWS], xb[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = h0 + i * HPR;
    xa[i] = xb[i] = make_uint2(0u, 0u);
    if (h < heads) {
      xa[i] = __ldg(reinterpret_cast<const uint2*>(src + h * D + ea));
      xb[i] = __ldg(reinterpret_cast<const uint2*>(src + h * D + eb));
    }
  }
  const bool bad_pos = pos < 0 || pos >= p.max_positions;
  const bool bad_slot = slot < -1 || slot >= p.num_slots;
  if ((bad_pos || bad_slot) && lane == 0)
    atomicOr(&g_rope_error, (bad_pos ? kErrBadPosition : 0u) | (bad_slot ? kErrBadSlot : 0u));
  if (bad_pos) return;                              // the whole token is skipped
  if (!is_q && (slot == -1 || bad_slot)) return;

  // where head h's elements go: q_out, or the slot's row of a pool
  const int64_t row0 = is_q ? t * p.q_heads : slot * p.kv_heads;
  if (is_v) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int h = h0 + i * HPR;
      if (h >= heads) continue;
      const int64_t at = (row0 + h) * D;
      if constexpr (FP8) {
        const uint64_t inv = f2_pack(p.v_inv, p.v_inv);
        uint8_t* dst = static_cast<uint8_t*>(p.v_cache) + at;
        *reinterpret_cast<uint32_t*>(dst + ea) =
            e4m3x4_of_f2(f2_mul(f2_of_bf16x2(xa[i].x), inv), f2_mul(f2_of_bf16x2(xa[i].y), inv));
        *reinterpret_cast<uint32_t*>(dst + eb) =
            e4m3x4_of_f2(f2_mul(f2_of_bf16x2(xb[i].x), inv), f2_mul(f2_of_bf16x2(xb[i].y), inv));
      } else {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.v_cache) + at;
        *reinterpret_cast<uint2*>(dst + ea) = xa[i];
        *reinterpret_cast<uint2*>(dst + eb) = xb[i];
      }
    }
    return;
  }

  const __nv_bfloat16* weight = is_q ? p.q_weight : p.k_weight;
  uint64_t wa[2], wb[2];  // weights of the two runs, two elements each
  wa[0] = wa[1] = wb[0] = wb[1] = f2_pack(1.f, 1.f);
  if (weight) {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(weight + ea));
    const uint2 b = __ldg(reinterpret_cast<const uint2*>(weight + eb));
    wa[0] = f2_of_bf16x2(a.x), wa[1] = f2_of_bf16x2(a.y);
    wb[0] = f2_of_bf16x2(b.x), wb[1] = f2_of_bf16x2(b.y);
  }
  // cosines and sines of pairs 4 hl .. 4 hl + 3
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turns) {
    const float* row = p.table + pos * p.rot_dim + 4 * hl;
    c = __ldg(reinterpret_cast<const float4*>(row));
    s = __ldg(reinterpret_cast<const float4*>(row + p.rot_dim / 2));
  }
  // apart:       y_a = x_a (w_a c) + x_b (-w_b s),  y_b = x_b (w_b c) + x_a (w_a s)
  // interleaved: y = x (w c) + swap(x) (swap(w) (-s, s)), pairs side by side
  uint64_t same_a[2], same_b[2], cross_a[2], cross_b[2];
  if constexpr (INTERLEAVED) {
    const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float lo, hi;
      same_a[i] = f2_mul(wa[i], f2_pack(cs[i], cs[i]));
      same_b[i] = f2_mul(wb[i], f2_pack(cs[2 + i], cs[2 + i]));
      f2_unpack(wa[i], lo, hi);
      cross_a[i] = f2_mul(f2_pack(hi, lo), f2_pack(-sn[i], sn[i]));
      f2_unpack(wb[i], lo, hi);
      cross_b[i] = f2_mul(f2_pack(hi, lo), f2_pack(-sn[2 + i], sn[2 + i]));
    }
  } else {
    const uint64_t cc[2] = {f2_pack(c.x, c.y), f2_pack(c.z, c.w)};
    const uint64_t ss[2] = {f2_pack(s.x, s.y), f2_pack(s.z, s.w)};
    const uint64_t neg = f2_pack(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      same_a[i] = f2_mul(wa[i], cc[i]);
      same_b[i] = f2_mul(wb[i], cc[i]);
      cross_a[i] = f2_mul(f2_mul(wb[i], ss[i]), neg);
      cross_b[i] = f2_mul(wa[i], ss[i]);
    }
  }

  // the heads' factors: 1 / rms, and 1 / scale for codes
  float inv[ROWS];
  const float unit_scale = is_q || !FP8 ? 1.f : p.k_inv;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) inv[i] = unit_scale;
  if (weight) {  // uniform over the warp
    float sum[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const uint64_t a0 = f2_of_bf16x2(xa[i].x), a1 = f2_of_bf16x2(xa[i].y);
      const uint64_t b0 = f2_of_bf16x2(xb[i].x), b1 = f2_of_bf16x2(xb[i].y);
      float lo, hi;
      f2_unpack(f2_fma(a0, a0, f2_fma(a1, a1, f2_fma(b0, b0, f2_mul(b1, b1)))), lo, hi);
      sum[i] = lo + hi;
    }
    if constexpr (ROWS == 4) {
      // four sums over LPH lanes at once: the lanes' halves, then quarters,
      // take over a part of the heads each, so that 9 shuffles do for 16
      const bool up = lane & (LPH / 2), side = lane & (LPH / 4);
      float k0 = up ? sum[2] : sum[0], k1 = up ? sum[3] : sum[1];
      k0 += __shfl_xor_sync(0xffffffffu, up ? sum[0] : sum[2], LPH / 2);
      k1 += __shfl_xor_sync(0xffffffffu, up ? sum[1] : sum[3], LPH / 2);
      float k = side ? k1 : k0;
      k += __shfl_xor_sync(0xffffffffu, side ? k0 : k1, LPH / 4);
#pragma unroll
      for (int o = LPH / 8; o > 0; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
      k = unit_scale * rsqrtf(k * (1.f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        inv[i] = __shfl_sync(0xffffffffu, k, (lane & ~(LPH - 1)) + (i >> 1) * (LPH / 2) +
                                                 (i & 1) * (LPH / 4));
    } else {
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
        inv[i] *= rsqrtf(sum[i] * (1.f / D) + p.eps);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = h0 + i * HPR;
    const uint64_t fa[2] = {f2_of_bf16x2(xa[i].x), f2_of_bf16x2(xa[i].y)};
    const uint64_t fb[2] = {f2_of_bf16x2(xb[i].x), f2_of_bf16x2(xb[i].y)};
    const uint64_t inv2 = f2_pack(inv[i], inv[i]);
    uint64_t ya[2], yb[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      uint64_t oa = fb[z], ob = fa[z];  // what the sines multiply
      if constexpr (INTERLEAVED) {
        float lo, hi;
        f2_unpack(fa[z], lo, hi);
        oa = f2_pack(hi, lo);
        f2_unpack(fb[z], lo, hi);
        ob = f2_pack(hi, lo);
      }
      // elements beyond the rotated ones have no partner: an infinity there
      // must not meet a sine of 0
      ya[z] = f2_mul(fa[z], same_a[z]);
      yb[z] = f2_mul(fb[z], same_b[z]);
      if (turns) {
        ya[z] = f2_fma(oa, cross_a[z], ya[z]);
        yb[z] = f2_fma(ob, cross_b[z], yb[z]);
      }
      ya[z] = f2_mul(ya[z], inv2);
      yb[z] = f2_mul(yb[z], inv2);
    }
    if (h >= heads) continue;
    const int64_t at = (row0 + h) * D;
    if (FP8 && !is_q) {
      uint8_t* dst = static_cast<uint8_t*>(p.k_cache) + at;
      *reinterpret_cast<uint32_t*>(dst + ea) = e4m3x4_of_f2(ya[0], ya[1]);
      *reinterpret_cast<uint32_t*>(dst + eb) = e4m3x4_of_f2(yb[0], yb[1]);
    } else {
      __nv_bfloat16* dst = (is_q ? p.q_out : static_cast<__nv_bfloat16*>(p.k_cache)) + at;
      *reinterpret_cast<uint2*>(dst + ea) = make_uint2(bf16x2_of_f2(ya[0]), bf16x2_of_f2(ya[1]));
      *reinterpret_cast<uint2*>(dst + eb) = make_uint2(bf16x2_of_f2(yb[0]), bf16x2_of_f2(yb[1]));
    }
  }
}

cudaError_t rope_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_rope_error);
}

unsigned read_rope_error(bool clear) {
  unsigned word = 0;
  if (cudaMemcpyFromSymbol(&word, g_rope_error, sizeof(word)) != cudaSuccess) return ~0u;
  if (clear) {
    const unsigned zero = 0;
    if (cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  }
  return word;
}

template <int D, bool INTERLEAVED, bool FP8, int ROWS>
static cudaError_t launch_rope_t(const QkRopeArgs& a, cudaStream_t stream) {
  constexpr int HPU = ROWS * (32 / (D / 8));
  const int64_t units = (a.q_heads + HPU - 1) / HPU + 2 * ((a.kv_heads + HPU - 1) / HPU);
  const int64_t blocks = (a.num_tokens * units * 32 + kRopeThreads - 1) / kRopeThreads;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  return launch_after_previous(qk_rope_append_kernel<D, INTERLEAVED, FP8, ROWS>,
                               dim3(unsigned(blocks)), dim3(kRopeThreads), 0, stream, a);
}

template <int D, bool INTERLEAVED, bool FP8>
static cudaError_t launch_rope_r(const QkRopeArgs& a, int num_sms, cudaStream_t stream) {
  // One head (two of 64) per warp spreads a few tokens over the SMs; four share
  // the angles, the weights and the shuffles once there is work enough.  Measured
  // on GB300, one / four, us: 64 q + 2 x 8 kv heads of 128: 1 token 1.48 / 1.74, 64
  // 1.93 / 1.95, 128 2.65 / 2.25, 2048 22.98 / 12.46; 16 + 2 x 4 heads of 64: 512
  // tokens 1.95 / 2.20, 1024 2.89 / 2.69.
  const int64_t rows = a.num_tokens * (a.q_heads + 2 * a.kv_heads) / (32 / (D / 8));
  return rows >= int64_t(num_sms) * 24 ? launch_rope_t<D, INTERLEAVED, FP8, 4>(a, stream)
                                       : launch_rope_t<D, INTERLEAVED, FP8, 1>(a, stream);
}

template <int D>
static cudaError_t launch_rope_d(const QkRopeArgs& a, int num_sms, cudaStream_t stream) {
  if (a.interleaved)
    return a.fp8 ? launch_rope_r<D, true, true>(a, num_sms, stream)
                 : launch_rope_r<D, true, false>(a, num_sms, stream);
  return a.fp8 ? launch_rope_r<D, false, true>(a, num_sms, stream)
               : launch_rope_r<D, false, false>(a, num_sms, stream);
}

cudaError_t launch_qk_rope_append(const QkRopeArgs& a, int d_head, int num_sms,
                                  cudaStream_t stream) {
  if (d_head == 128) return launch_rope_d<128>(a, num_sms, stream);
  if (d_head == 64) return launch_rope_d<64>(a, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pkv
