// What the kernels of w8_route.hip, w8_moe_layer.hip and w8_rows.hip need of the
// device language beside hip/hip_runtime.h, included in front of them.  LDS
// variables are one for all threads (static); the accesses of a wavefront to its
// own LDS are in order, which the kernels rely on behind a signal fence or a wave
// barrier: there its lanes wait for each other.
#pragma once
#include <hip/hip_runtime.h>

#undef __shared__
#define __shared__ static

namespace emu {
inline void wave_sync() {
  const unsigned w = 0;
  wave_op(kSync, &w, 4);
}
// to the nearest E4M3FN code, ties to even; finite values up to 448 (NaN: 0x7F)
inline unsigned e4m3_code(float f) {
  const unsigned sign = __builtin_bit_cast(unsigned, f) >> 31 << 7;
  const double v = std::fabs((double)f);
  if (v != v) return sign | 0x7F;
  unsigned best = 0;
  double at = 1e30;
  for (unsigned c = 0; c < 127; ++c) {
    const double d = std::fabs(e4m3((uint8_t)c) - v);
    if (d < at || (d == at && !(c & 1))) best = c, at = d;
  }
  return sign | best;
}
inline int cvt_pk_fp8(float a, float b, int old, bool hi) {
  const unsigned pair = e4m3_code(a) | e4m3_code(b) << 8;
  return (int)(hi ? ((unsigned)old & 0xFFFFu) | pair << 16 : ((unsigned)old & 0xFFFF0000u) | pair);
}
template <class T>
inline T atomic_add(T* p, T v) {
  const T old = *p;
  *p += v;
  return old;
}
inline unsigned lanes_below(unsigned half, unsigned mask, unsigned base) {
  const int lane = m().current % 64 - 32 * (int)half;
  const unsigned below = lane >= 32 ? ~0u : lane <= 0 ? 0u : (1u << lane) - 1;
  return base + __builtin_popcount(mask & below);
}
}  // namespace emu

#undef __builtin_amdgcn_cvt_pk_fp8_f32
#define __builtin_amdgcn_cvt_pk_fp8_f32(a, b, old, hi) emu::cvt_pk_fp8(a, b, old, hi)
#define __builtin_amdgcn_exp2f(x) exp2f(x)
#define __builtin_amdgcn_rcpf(x) (1.0f / (x))
#define __builtin_amdgcn_mbcnt_lo(mask, base) emu::lanes_below(0, mask, base)
#define __builtin_amdgcn_mbcnt_hi(mask, base) emu::lanes_below(1, mask, base)
#define __atomic_signal_fence(order) emu::wave_sync()
#define __builtin_amdgcn_wave_barrier() emu::wave_sync()
#define __hip_atomic_store(p, v, order, scope) ((void)(*(p) = (v)))
#define __hip_atomic_load(p, order, scope) (*(p))
#define atomicAdd(p, v) emu::atomic_add(p, v)
#define atomicMax(p, v) ((void)(*(p) = max(*(p), v)))
#define atomicOr(p, v) ((void)(*(p) |= (v)))
inline int __popc(unsigned v) { return __builtin_popcount(v); }
inline int __popcll(unsigned long long v) { return __builtin_popcountll(v); }
inline unsigned __umulhi(unsigned a, unsigned b) { return (unsigned)((unsigned long long)a * b >> 32); }
// (named in kernels of the shared headers that do not run here)
float __shfl(float, int, int);
float __shfl_xor(float, int, int = 64);
#define __builtin_amdgcn_global_load_lds(...) ((void)0)
inline hipError_t hipGetLastError() { return hipSuccess; }
