// Row operators of the Block_FP8 layer for any token count: the 1 x 128
// quantizer with the gated activation in front of it, and the residual
// update with its norms.  Both read every input once and write every output
// once; HBM bandwidth bounds them on many rows and launch latency on few.
#include <type_traits>

#include "w8_block.hpp"
#include "w8_device.hpp"

namespace w8 {
namespace {

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

// Sum over the 64 lanes of a wavefront, in a fixed order.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_move<0xB1>(v);
  v += dpp_move<0x4E>(v);
  v += dpp_move<0x141>(v);
  v += dpp_move<0x140>(v);
  const int b = __builtin_bit_cast(int, v);
  const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
  const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
  const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
  const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
  return (r0 + r1) + (r2 + r3);
}

// fp32 -> bf16, round to nearest even; a NaN stays a NaN.
__device__ __forceinline__ unsigned bf16_bits(float f) {
  return abs_bits(f) > 0x7F800000u ? 0x7FC0u : (unsigned)bf16_rne(f);
}

__device__ __forceinline__ void unpack8(v4u v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(v[i]);
    f[2 * i + 1] = bf16_hi(v[i]);
  }
}

// Eight values of a row of D from element k on, 16 bytes a load at the
// elements' own alignment.  Past D - 8 the row's last eight are loaded, so that
// no load waits for a condition, and trim8() moves them into place (a load for
// each element of a short chunk took 2235 x 1871 from 12 to 20 us).
__device__ __forceinline__ v4u load8_bf16(const uint16_t* row, int k, int D) {
  v4u v;
  __builtin_memcpy(&v, row + min(k, D - 8), 16);
  return v;
}
struct Raw8 {
  float f[8];
};
__device__ __forceinline__ Raw8 load8_f32(const float* row, int k, int D) {
  Raw8 v;
  __builtin_memcpy(v.f, row + min(k, D - 8), 32);
  return v;
}
// The eight values from k on of what load8 loaded: zeros past the row's end.
__device__ __forceinline__ void trim8(v4u& v, int k, int D) {
  const int s = k - (D - 8);
  if (s <= 0) return;
  unsigned long long lo = v[0] | (unsigned long long)v[1] << 32;
  unsigned long long hi = v[2] | (unsigned long long)v[3] << 32;
  const int b = 16 * (s & 3);
  if (s & 4) {
    lo = hi;
    hi = 0;
  }
  lo = lo >> b | (b ? hi << (64 - b) : 0);
  hi >>= b;
  v = s < 8 ? v4u{(unsigned)lo, (unsigned)(lo >> 32), (unsigned)hi, (unsigned)(hi >> 32)}
            : v4u{0u, 0u, 0u, 0u};
}
__device__ __forceinline__ void trim8(Raw8& v, int k, int D) {
  const int s = k - (D - 8);
  if (s <= 0) return;
#pragma unroll
  for (int by = 4; by; by >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) v.f[i] = s & by ? (i + by < 8 ? v.f[i + by] : 0.0f) : v.f[i];
#pragma unroll
  for (int i = 0; i < 8; ++i) v.f[i] = s < 8 ? v.f[i] : 0.0f;
}
// The same of a row of fewer than eight elements.
__device__ __forceinline__ v4u short8_bf16(const uint16_t* row, int k, int D) {
  v4u v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (k + i < D) v[i >> 1] |= (unsigned)row[k + i] << (16 * (i & 1));
  return v;
}
__device__ __forceinline__ Raw8 short8_f32(const float* row, int k, int D) {
  Raw8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v.f[i] = k + i < D ? row[k + i] : 0.0f;
  return v;
}
__device__ __forceinline__ void store8_bf16(uint16_t* p, int n, const float* f) {
  if (n >= 8) {
    v4u v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = bf16_bits(f[2 * i]) | (bf16_bits(f[2 * i + 1]) << 16);
    __builtin_memcpy(p, &v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint16_t)bf16_bits(f[i]);
  }
}
__device__ __forceinline__ void store8_f32(float* p, int n, const float* f) {
  if (n >= 8) {
    __builtin_memcpy(p, f, 32);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = f[i];
  }
}
__device__ __forceinline__ void store8_codes(uint8_t* p, int n, v2u v) {
  if (n >= 8) {
    __builtin_memcpy(p, &v, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)(v[i >> 2] >> (8 * (i & 3)));
  }
}

// Codes of eight values of a 1 x 128 group whose 16 lanes call together; *s
// is the scale of the group times `factor` (1 for zeros).  A group that holds a
// NaN or an infinity gets a NaN or infinite scale, so that it stays non-finite
// when dequantized.
__device__ __forceinline__ v2u encode_group(float* f, float* scale, float factor = 1.0f) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(f[i]));
  m = seg16_umax(m);
  const float s = act_scale<false>(__uint_as_float(m));
  *scale = m ? s * factor : 1.0f;
  const float r = act_recip(s);
  if (r != 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = act_quot(f[i], s, r);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] / s;
  }
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

// ---------------------------------------------------------------- quantize --
// 16 lanes take a group, each lane eight values; a workgroup takes 16 groups
// and strides over the rest.  Bound by HBM on many rows (32768 x 768 gated:
// 27.6 us, 4.6 TB/s; a copy reaches 4.8) and by the launch on few (33 x 2048:
// 2.6 us).
constexpr int kQThreads = 256;

template <bool GATED>
__global__ __launch_bounds__(kQThreads) void block_quantize_kernel(BlockQuantArgs a) {
  const int j = threadIdx.x & 15;
  for (unsigned id = blockIdx.x * (kQThreads / 16) + (threadIdx.x >> 4); id < a.groups;
       id += gridDim.x * (kQThreads / 16)) {
    // (groups < 2^31: the quotient by a multiplication, exact for such ids)
    const unsigned row = a.shift < 0 ? id : __umulhi(id, a.magic) >> a.shift;
    const long long m = row;
    const int k = (int)(id - row * a.G) * kGroup + 8 * j;
    const int n = a.K - k;
    float f[8];
    // (K is a multiple of 8: a chunk is whole or past the end)
    v4u x = load8_bf16(a.x + m * a.ldx, k, a.K);
    if (n <= 0) x = v4u{0u, 0u, 0u, 0u};
    unpack8(x, f);
    if (GATED) {
      float g[8];
      v4u y = load8_bf16(a.gate + m * a.ldg, k, a.K);
      if (n <= 0) y = v4u{0u, 0u, 0u, 0u};
      unpack8(y, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= silu(g[i]);
    }
    float s;
    const v2u q = encode_group(f, &s);
    if (j == 0) a.sx[id] = s;
    store8_codes(a.xq + m * a.ldq + k, n, q);
  }
}

// -------------------------------------------------------------------- norm --
// One row by the waves of a workgroup (ONE_WAVE: four rows, a wave each), NC
// chunks of eight values a lane, kept in registers between the two norms, so
// that every input is read once.  Sums of squares are fp32, in a fixed order.
// Bound by HBM on many rows (8192 x 5120, fp32 residual, post norm, gate rows:
// 111 us, 5.3 TB/s) and on one by its chain of load, sum, sum and store (1 x
// 7168 to codes: 3.9 us).
template <bool ONE_WAVE>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if (ONE_WAVE) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.0f;
  for (unsigned w = 0; w < blockDim.x / 64; ++w) t += red[w];
  return t;
}

template <bool ONE_WAVE, int NC, bool RF32, bool RAGGED>
__global__ __launch_bounds__(ONE_WAVE ? 256 : 1024) void residual_norm_kernel(NormArgs a) {
  __shared__ float red[2][16];
  const int T = ONE_WAVE ? 64 : blockDim.x;
  const int t = ONE_WAVE ? threadIdx.x & 63 : threadIdx.x;
  const long long row =
      ONE_WAVE ? (long long)blockIdx.x * 4 + (threadIdx.x >> 6) : (long long)blockIdx.x;
  if (ONE_WAVE && row >= a.M) return;  // (no barrier with one wave per row)
  const uint16_t* y = a.y + row * a.ldy;
  const void* res = RF32 ? (const void*)(static_cast<const float*>(a.residual) + row * a.ldr)
                         : (const void*)(static_cast<const uint16_t*>(a.residual) + row * a.ldr);
  const uint16_t* gate = a.gate ? a.gate + row * a.ldg : nullptr;
  const bool is_short = RAGGED && ONE_WAVE && a.D < 8;
  auto load = [&](const uint16_t* p, int c) {
    const int k = 8 * (t + c * T);
    return is_short ? short8_bf16(p, k, a.D) : load8_bf16(p, k, a.D);
  };
  auto load_f32 = [&](const float* p, int c) {
    const int k = 8 * (t + c * T);
    return is_short ? short8_f32(p, k, a.D) : load8_f32(p, k, a.D);
  };
  // (RAGGED: D is no multiple of 8)
  auto trim = [&](auto& v, int c) {
    if (RAGGED && !is_short) trim8(v, 8 * (t + c * T), a.D);
  };
  float h[NC][8], b[NC][8];
  // the factors too are loaded up front, where there are registers for that
  // (four chunks a lane: at their use, from L2 for all rows but the first)
  constexpr bool EARLY = NC < 4;
  constexpr int NF = EARLY ? NC : 1;
  typedef std::conditional_t<RF32, Raw8, v4u> Residual;
  v4u yv[NC] = {}, g[NF] = {}, pw[NF] = {}, w[NF] = {};
  Residual rv[NC] = {};
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (8 * (t + c * T) >= a.D) continue;
    yv[c] = load(y, c);
    if constexpr (RF32)
      rv[c] = load_f32(static_cast<const float*>(res), c);
    else
      rv[c] = load(static_cast<const uint16_t*>(res), c);
    if constexpr (EARLY) {
      if (gate) g[c] = load(gate, c);
      if (a.post_w) pw[c] = load(a.post_w, c);
      w[c] = load(a.w, c);
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    trim(yv[c], c);
    unpack8(yv[c], b[c]);
    trim(rv[c], c);
    if constexpr (RF32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = rv[c].f[i];
    } else {
      unpack8(rv[c], h[c]);
    }
  }
  auto factor = [&](const v4u* held, const uint16_t* p, int c) {
    v4u v;
    if constexpr (EARLY) {
      v = held[c];
    } else {
      v = v4u{0u, 0u, 0u, 0u};
      if (8 * (t + c * T) < a.D) v = load(p, c);
    }
    trim(v, c);
    return v;
  };
  if (a.post_w) {
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(b[c][i], b[c][i], ss);
    const float r = 1.0f / sqrtf(row_sum<ONE_WAVE>(ss, red[0]) / (float)a.D + a.eps);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float p[8];
      unpack8(factor(pw, a.post_w, c), p);
#pragma unroll
      for (int i = 0; i < 8; ++i) b[c][i] *= r * p[i];
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float gf[8];
    if (gate) unpack8(factor(g, gate, c), gf);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (gate) b[c][i] *= gf[i];
      h[c][i] = __builtin_fmaf(a.scale, b[c][i], h[c][i]);
      ss = __builtin_fmaf(h[c][i], h[c][i], ss);
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int k = 8 * (t + c * T), n = a.D - k;
    if (RF32)
      store8_f32(static_cast<float*>(a.h) + row * a.ldh + k, n, h[c]);
    else
      store8_bf16(static_cast<uint16_t*>(a.h) + row * a.ldh + k, n, h[c]);
  }
  const float r = 1.0f / sqrtf(row_sum<ONE_WAVE>(ss, red[1]) / (float)a.D + a.eps);
  const int G = (a.D + kGroup - 1) / kGroup;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int k = 8 * (t + c * T), n = a.D - k;
    float wf[8];
    unpack8(factor(w, a.w, c), wf);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[c][i] *= wf[i];
    if (a.z) {
      float z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = h[c][i] * r;
      store8_bf16(a.z + row * a.ldz + k, n, z);
    }
    if (a.zq) {  // 16 consecutive lanes hold one group
      // The row's factor r leaves the codes alone and goes into the scale (one
      // rounding less a code), unless it is 0, infinite or NaN: then it decides
      // what the values are, zeros among them.
      const bool apart = r > 0.0f && r < __builtin_inff();
      if (!apart) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] *= r;
      }
      float s;
      const v2u q = encode_group(h[c], &s, apart ? r : 1.0f);
      if ((t & 15) == 0 && n > 0) a.sz[row * G + k / kGroup] = s;
      store8_codes(a.zq + row * a.ldq + k, n, q);
    }
  }
}

template <bool ONE_WAVE, int NC>
hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  // as many waves as the row has chunks for
  const unsigned threads = ONE_WAVE ? 256u : (unsigned)((a.D + 512 * NC - 1) / (512 * NC)) * 64u;
  const dim3 grid((unsigned)(ONE_WAVE ? (a.M + 3) / 4 : a.M)), block(threads);
  const auto kernel = a.D % 8 ? a.residual_fp32 ? residual_norm_kernel<ONE_WAVE, NC, true, true>
                                                : residual_norm_kernel<ONE_WAVE, NC, false, true>
                      : a.residual_fp32 ? residual_norm_kernel<ONE_WAVE, NC, true, false>
                                        : residual_norm_kernel<ONE_WAVE, NC, false, false>;
  return launch_kernel(kernel, grid, block, 0, s, a);
}

}  // namespace

hipError_t launch_block_quantize(BlockQuantArgs a, hipStream_t s) {
  // id / G = umulhi(id, magic) >> shift for id < 2^31, with magic the
  // reciprocal 2^(32 + shift) / G rounded up, 2^shift < G <= 2^(shift + 1)
  a.shift = -1;
  if (a.G > 1) {
    a.shift = 0;
    while ((2u << a.shift) < a.G) ++a.shift;
    a.magic = (unsigned)(((1ull << (32 + a.shift)) + a.G - 1) / a.G);
  }
  const long long blocks = ((long long)a.groups + kQThreads / 16 - 1) / (kQThreads / 16);
  const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20))), block(kQThreads);
  return launch_kernel(a.gate ? block_quantize_kernel<true> : block_quantize_kernel<false>, grid,
                       block, 0, s, a);
}

hipError_t launch_residual_norm(const NormArgs& a, hipStream_t s) {
  // One chunk a lane has the shortest chain of a single row (1 x 7168: 4.0 us,
  // two chunks 4.2, four 5.5) and the most loads in flight on fp32 residuals
  // (8192 x 5120: 111.0 us, 112.1, 122.9); many long bf16 rows move too few
  // bytes a lane that way (8192 x 5120: 63.1 us, 57.2, 63.6; 8192 x 2048: 27.3,
  // 25.9, 30.6).
  if (a.D <= 512) return launch_norm<true, 1>(a, s);
  if (a.D <= 8192 && (a.residual_fp32 || a.M < 512 || a.D < 2048))
    return launch_norm<false, 1>(a, s);
  if (a.D <= 16384) return launch_norm<false, 2>(a, s);
  return launch_norm<false, 4>(a, s);
}

}  // namespace w8
