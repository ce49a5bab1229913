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
// Bound by memory: each q, k, v element is read once and written once, ~8
// flops each.  A lane holds 8 consecutive elements (one 16-byte load), d / 8
// lanes a head, so a norm is log2(d / 8) shuffles and a rotation partner sits
// in the same lane (interleaved) or rot / 16 lanes away (one packed shuffle of
// the raw bf16 values; the partner's weight is loaded instead of its product).
// A warp takes kRows row slots of one token's q, k and v heads laid end to
// end, so the token's angles and the weights are loaded once for all of them.
#include <cuda_fp8.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

static __device__ unsigned g_rope_error = 0;

constexpr int kRopeThreads = 128;

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf16_lo_to_f32(v.x), f[1] = bf16_hi_to_f32(v.x);
  f[2] = bf16_lo_to_f32(v.y), f[3] = bf16_hi_to_f32(v.y);
  f[4] = bf16_lo_to_f32(v.z), f[5] = bf16_hi_to_f32(v.z);
  f[6] = bf16_lo_to_f32(v.w), f[7] = bf16_hi_to_f32(v.w);
}

__device__ __forceinline__ uint4 pack8_bf16(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return (lo & 0xffffu) | (hi << 16);
}

__device__ __forceinline__ uint2 pack8_e4m3(const float (&f)[8], float inv) {
  return make_uint2(e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                    e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}

// ROWS: row slots in flight per lane.
template <int D, bool INTERLEAVED, bool FP8, int ROWS>
__global__ void __launch_bounds__(kRopeThreads)
qk_rope_append_kernel(const QkRopeArgs p) {
  griddep_wait();  // inputs may have been written by the previous kernel in the stream
  constexpr int LPH = D / 8;       // lanes per head
  constexpr int HPR = 32 / LPH;    // heads per row slot
  constexpr int HPU = ROWS * HPR;  // heads per warp
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t(blockIdx.x) * kRopeThreads + threadIdx.x) >> 5;
  const int heads = p.q_heads + 2 * p.kv_heads;
  const int units = (heads + HPU - 1) / HPU;  // warps per token
  const int64_t t = unit / units;
  if (t >= p.num_tokens) return;
  const int h0 = int(unit - t * units) * HPU + lane / LPH;
  const int hl = lane % LPH;  // this lane's 8 elements: 8 hl ..

  const int64_t pos = __ldg(p.positions + t);
  const int64_t slot = __ldg(p.slot_mapping + t);
  uint4 x[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = h0 + i * HPR;
    const uint4* src = nullptr;
    if (h < p.q_heads)
      src = p.q + t * p.q_stride_vec + int64_t(h) * LPH;
    else if (h < p.q_heads + p.kv_heads)
      src = p.k + t * p.k_stride_vec + int64_t(h - p.q_heads) * LPH;
    else if (h < heads)
      src = p.v + t * p.v_stride_vec + int64_t(h - p.q_heads - p.kv_heads) * LPH;
    x[i] = src ? __ldg(src + hl) : make_uint4(0u, 0u, 0u, 0u);
  }
  const bool bad_pos = pos < 0 || pos >= p.max_positions;
  const bool bad_slot = slot < -1 || slot >= p.num_slots;
  if ((bad_pos || bad_slot) && lane == 0)
    atomicOr(&g_rope_error, (bad_pos ? kErrBadPosition : 0u) | (bad_slot ? kErrBadSlot : 0u));
  if (bad_pos) return;  // the whole token is skipped

  // angles of this lane's elements (or pairs)
  const int half = p.rot_dim / 2;
  const bool turns = 8 * hl < p.rot_dim;
  const bool second = !INTERLEAVED && 8 * hl >= half;
  constexpr int NC = INTERLEAVED ? 4 : 8;
  float c[NC], s[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) c[i] = 1.f, s[i] = 0.f;
  if (turns) {
    const float* row = p.table + pos * p.rot_dim +
                       (INTERLEAVED ? 4 * hl : (second ? 8 * hl - half : 8 * hl));
#pragma unroll
    for (int i = 0; i < NC; i += 4) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + i));
      const float4 b = __ldg(reinterpret_cast<const float4*>(row + half + i));
      c[i] = a.x, c[i + 1] = a.y, c[i + 2] = a.z, c[i + 3] = a.w;
      s[i] = b.x, s[i + 1] = b.y, s[i + 2] = b.z, s[i + 3] = b.w;
    }
  }
  const int reach = half / 8;  // lanes between the halves of a pair
  const int partner = (turns && !INTERLEAVED) ? (second ? lane - reach : lane + reach) : lane;
  const int pl = partner % LPH;
  const uint4 one = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  uint4 qw = one, kw = one, qwp = one, kwp = one;
  if (p.q_weight) qw = __ldg(p.q_weight + hl), qwp = __ldg(p.q_weight + pl);
  if (p.k_weight) kw = __ldg(p.k_weight + hl), kwp = __ldg(p.k_weight + pl);

#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = h0 + i * HPR;
    const bool is_q = h < p.q_heads;
    const bool is_k = !is_q && h < p.q_heads + p.kv_heads;
    float f[8];
    unpack8(x[i], f);
    float inv = 1.f;
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (is_q ? p.q_weight != nullptr : (is_k && p.k_weight != nullptr))
      inv = rsqrtf(ss * (1.f / D) + p.eps);
    uint4 other = x[i];
    if constexpr (!INTERLEAVED) {
      other.x = __shfl_sync(0xffffffffu, x[i].x, partner);
      other.y = __shfl_sync(0xffffffffu, x[i].y, partner);
      other.z = __shfl_sync(0xffffffffu, x[i].z, partner);
      other.w = __shfl_sync(0xffffffffu, x[i].w, partner);
    }
    float y[8];
    if (is_q || is_k) {
      float w[8];
      unpack8(is_q ? qw : kw, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = f[e] * inv * w[e];
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[2 * e] = f[2 * e] * c[e] - f[2 * e + 1] * s[e];
          y[2 * e + 1] = f[2 * e + 1] * c[e] + f[2 * e] * s[e];
        }
      } else {
        float g[8];
        unpack8(other, g);
        unpack8(is_q ? qwp : kwp, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          g[e] = g[e] * inv * w[e];
          y[e] = f[e] * c[e] + (second ? g[e] : -g[e]) * s[e];
        }
        if (!turns) {  // g is the element itself: keep an infinity out of 0 * inf
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = f[e];
        }
      }
      if (INTERLEAVED && !turns) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = f[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = f[e];
    }
    if (is_q) {
      p.q_out[(t * p.q_heads + h) * LPH + hl] = pack8_bf16(y);
    } else if (h < heads && slot != -1 && !bad_slot) {
      const int kvh = is_k ? h - p.q_heads : h - p.q_heads - p.kv_heads;
      void* pool = is_k ? p.k_cache : p.v_cache;
      const int64_t at = (slot * p.kv_heads + kvh) * LPH + hl;
      if constexpr (FP8)
        static_cast<uint2*>(pool)[at] = pack8_e4m3(y, is_k ? p.k_inv : p.v_inv);
      else
        static_cast<uint4*>(pool)[at] = is_k ? pack8_bf16(y) : x[i];
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
  const int64_t units = (a.q_heads + 2 * a.kv_heads + HPU - 1) / HPU;
  const int64_t blocks = (a.num_tokens * units * 32 + kRopeThreads - 1) / kRopeThreads;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  return launch_after_previous(qk_rope_append_kernel<D, INTERLEAVED, FP8, ROWS>,
                               dim3(unsigned(blocks)), dim3(kRopeThreads), 0, stream, a);
}

template <int D, bool INTERLEAVED, bool FP8>
static cudaError_t launch_rope_r(const QkRopeArgs& a, int num_sms, cudaStream_t stream) {
  // one row slot per warp spreads a few tokens over the SMs; four share the
  // angles once there are warps enough to fill them
  const int64_t rows = a.num_tokens * (a.q_heads + 2 * a.kv_heads) / (32 / (D / 8));
  return rows >= int64_t(num_sms) * 64 ? launch_rope_t<D, INTERLEAVED, FP8, 4>(a, stream)
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
