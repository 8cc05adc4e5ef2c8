// Device-side steps shared by the row operators and the MoE layer: maxima that
// keep a NaN, the codes of fp32 values, the gated activation's silu.
#pragma once
#include "w8_device.hpp"

namespace w8 {

// The bits of |v|: ordered like the magnitudes for finite values, infinities
// above them and NaN above those, so an unsigned maximum keeps a NaN where
// fmaxf would drop it.
__device__ __forceinline__ unsigned abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

template <int CTRL>
__device__ __forceinline__ unsigned dpp_move_u(unsigned v) {
  return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

// Maximum over aligned segments of 16 lanes.
__device__ __forceinline__ unsigned seg16_umax(unsigned v) {
  v = max(v, dpp_move_u<0xB1>(v));
  v = max(v, dpp_move_u<0x4E>(v));
  v = max(v, dpp_move_u<0x141>(v));
  v = max(v, dpp_move_u<0x140>(v));
  return v;
}

// Maximum over the 64 lanes of a wavefront.
__device__ __forceinline__ unsigned wave_umax(unsigned v) {
  v = seg16_umax(v);
  const unsigned r0 = __builtin_amdgcn_readlane((int)v, 0);
  const unsigned r1 = __builtin_amdgcn_readlane((int)v, 16);
  const unsigned r2 = __builtin_amdgcn_readlane((int)v, 32);
  const unsigned r3 = __builtin_amdgcn_readlane((int)v, 48);
  return max(max(r0, r1), max(r2, r3));
}

// fp32 -> bf16, round to nearest even; a NaN stays a NaN.
__device__ __forceinline__ unsigned bf16_bits(float f) {
  return abs_bits(f) > 0x7F800000u ? 0x7FC0u : (unsigned)bf16_rne(f);
}

// Codes of eight values for the scale s; r = act_recip(s).
template <bool INT8>
__device__ __forceinline__ v2u encode_values(float* f, float s, float r) {
  if (r != 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = act_quot(f[i], s, r);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] / s;
  }
  if (INT8) return v2u{i8_pack4(f[0], f[1], f[2], f[3]), i8_pack4(f[4], f[5], f[6], f[7])};
  return v2u{e4m3_pack4(f[0], f[1], f[2], f[3]), e4m3_pack4(f[4], f[5], f[6], f[7])};
}

// g * sigmoid(g) = g / d, d = 1 + exp(-g).  exp(-g) = 2^t with t = -g log2(e)
// taken as a rounded product and its remainder, which keeps the exponential's
// relative error at a few 2^-24 for every g (the rounded product alone loses
// |t| 2^-25 of it); the quotient from the reciprocal with one correction.
__device__ __forceinline__ float silu(float g) {
  const float hi = g * -0x1.715476p+0f;
  const float lo = __builtin_fmaf(g, -0x1.715476p+0f, -hi) - g * 0x1.4ae0cp-26f;
  const float e = __builtin_amdgcn_exp2f(hi);
  const float d = 1.0f + __builtin_fmaf(e, 0x1.62e43p-1f * lo, e);
  const float r = __builtin_amdgcn_rcpf(d);
  const float q = g * r;
  const float s = __builtin_fmaf(__builtin_fmaf(-q, d, g), r, q);
  if (hi > 126.0f) {
    // d is 2^hi to every bit and its reciprocal, below 2^-126, would come out
    // as 0: g 2^-hi, the power with 64 more in its exponent
    const float p = __builtin_amdgcn_exp2f(64.0f - hi);
    return p == 0.0f ? g * 0.0f : g * __builtin_fmaf(p, -0x1.62e43p-1f * lo, p) * 0x1p-64f;
  }
  return s;
}

}  // namespace w8
