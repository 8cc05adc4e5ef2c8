// The experts of a few tokens as a whole, in two launches:
//
//   up    a = x W1_e^T for the tokens of expert e, gate and up halves;
//         h = silu(a_gate) a_up in fp32, and its maxima over 16 columns
//   down  hq = codes of h in the format; p = hq W2_e^T;
//         y[t] = sum_j weights[t, j] p[t, j], by the last workgroup of a column
//         tile to arrive
//
// The weights' bytes are nearly all that a launch moves, so every workgroup
// streams its own piece of one expert's weights into MFMA registers, as the
// small-M GEMM does (A = weights, B = tokens: a lane's accumulators belong to
// one token).  Which experts have tokens, and which tokens, every workgroup
// finds for itself from the T x topk choices, so a launch needs no lists and
// reads no weights of an expert without tokens.
#include "w8_block.hpp"
#include "w8_gemm.hpp"
#include "w8_route.hpp"
#include "w8_values.hpp"

namespace w8 {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kMaxEntries = kLayerTokens * kMaxTopk;

// The choices of a launch in LDS: which experts have tokens, and the tokens of
// this workgroup's.
struct Choices {
  int ids[kMaxEntries];                // (-1: no expert of this call's)
  unsigned set[kMaxExperts / 32];      // experts with tokens
  int entry[kLayerTokens];          // first entry of each of the expert's tokens
};
struct Expert {
  int e;       // -1: fewer experts have tokens
  int tokens;  // of the expert
  int active;  // experts with tokens
};

// The slot-th expert that has tokens, in expert order; every wave computes it.
__device__ __forceinline__ Expert find_expert(const MoeLayerArgs& a, int slot, Choices& c) {
  const int lane = threadIdx.x & 63;
  if (threadIdx.x < kMaxExperts / 32) c.set[threadIdx.x] = 0u;
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * a.topk; i += kThreads) {
    const int id = a.experts[i];
    const bool on = (unsigned)id < (unsigned)a.E;
    c.ids[i] = on ? id : -1;
    if (on) atomicOr(&c.set[id >> 5], 1u << (id & 31));
  }
  __syncthreads();
  const unsigned word = lane < kMaxExperts / 32 ? c.set[lane] : 0u;
  const int upto = wave_scan(__popc(word));
  Expert x{-1, 0, __builtin_amdgcn_readlane(upto, 63)};
  const unsigned long long past = __ballot(upto > slot);
  if (past) {
    const int l = __builtin_ctzll(past);
    unsigned bits = __builtin_amdgcn_readlane((int)word, l);
    for (int i = l ? __builtin_amdgcn_readlane(upto, l - 1) : 0; i < slot; ++i) bits &= bits - 1;
    x.e = 32 * l + __builtin_ctz(bits);
    int first = -1;
    if (lane < a.T)
      for (int j = a.topk - 1; j >= 0; --j)
        if (c.ids[lane * a.topk + j] == x.e) first = lane * a.topk + j;
    const unsigned long long mine = __ballot(first >= 0);
    x.tokens = __popcll(mine);
    if (threadIdx.x < 64 && first >= 0) c.entry[__popcll(mine & ((1ull << lane) - 1))] = first;
  }
  __syncthreads();
  return x;
}

// The entry whose outputs serve entry i: the first of its token with the same
// expert.
__device__ __forceinline__ int served_by(const Choices& c, int i, int t, int topk) {
  int at = t * topk;
  while (c.ids[at] != c.ids[i]) ++at;
  return at;
}

// Accumulates the products of K-steps [la, lb) of NB blocks of 16 weight rows
// with MB blocks of 16 token rows.  weights(j, k), tokens(b, k): operands of
// step k, tails with zeros past K; scale(j, b, k): the Block_FP8 factor.  The
// steps up to kfull are whole.  Stages of U steps alternate between two
// register sets, the loads of the next in flight while one is multiplied; the
// first may begin before la, with zeros there, so that the loop has no
// conditions.
template <int FMT, int NB, int MB, int U, class W, class X, class S, class WT, class XT>
__device__ __forceinline__ void products(typename Traits<FMT>::Acc (&acc)[MB][NB], int la, int lb,
                                         int kfull, W weights, X tokens, S scale, WT weights_tail,
                                         XT tokens_tail) {
  typedef typename Traits<FMT>::Frag Frag;
  typedef typename Traits<FMT>::Acc Acc;
  constexpr bool BLOCK = FMT == BLOCK_FP8;
  struct Stage {
    Frag w[U][NB], x[U][MB];
    float sc[BLOCK ? U : 1][MB][NB];
  };
  auto load = [&](Stage& st, int k0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = max(k0 + u, la);
#pragma unroll
      for (int j = 0; j < NB; ++j) st.w[u][j] = weights(j, k);
#pragma unroll
      for (int b = 0; b < MB; ++b) st.x[u][b] = tokens(b, k);
      if constexpr (BLOCK) {
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int j = 0; j < NB; ++j) st.sc[u][b][j] = scale(j, b, k);
      }
    }
  };
  auto multiply = [&](const Frag& w, const Frag& x, Acc& c, float sc) {
    if constexpr (BLOCK) {
      const Acc p = mma<FMT, 1>(w, x, Acc{0, 0, 0, 0});
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = __builtin_fmaf(p[i], sc, c[i]);
    } else {
      c = mma<FMT, 1>(w, x, c);
    }
  };
  auto run = [&](const Stage& st, int k0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const Frag zero = {};
        const Frag w = k0 + u < la ? zero : st.w[u][j];
#pragma unroll
        for (int b = 0; b < MB; ++b)
          multiply(w, st.x[u][b], acc[b][j], BLOCK ? st.sc[u][b][j] : 0.0f);
      }
  };
  const int lfull = min(lb, kfull);
  const int ns = (max(lfull - la, 0) + U - 1) / U, k0 = lfull - ns * U;
  Stage A, B;
  if (ns > 0) load(A, k0);
  if (ns > 1) load(B, k0 + U);
  if (ns == 1) {
    run(A, k0);
  } else if (ns > 1) {
    run(A, k0);
    int s = 1;  // B holds stage s
    for (; s + 2 <= ns - 1; s += 2) {
      load(A, k0 + (s + 1) * U);
      run(B, k0 + s * U);
      load(B, k0 + (s + 2) * U);
      run(A, k0 + (s + 1) * U);
    }
    if (s + 1 <= ns - 1) {
      load(A, k0 + (s + 1) * U);
      run(B, k0 + s * U);
      run(A, k0 + (s + 1) * U);
    } else {
      run(B, k0 + s * U);
    }
  }
  if constexpr (!BLOCK) {  // (Block_FP8's K is whole steps)
    if (lb > kfull && la < lb) {
      Frag x[MB];
#pragma unroll
      for (int b = 0; b < MB; ++b) x[b] = tokens_tail(b);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const Frag w = weights_tail(j);
#pragma unroll
        for (int b = 0; b < MB; ++b) multiply(w, x[b], acc[b][j], 0.0f);
      }
    }
  }
}

// The wave's first fragment (PACKED) or row of 16 weight rows from row n.
template <int FMT, bool PACKED>
__device__ __forceinline__ const uint8_t* weight_rows(const uint8_t* w, long long ld, int ksteps,
                                                      int n) {
  const int lane = threadIdx.x & 63;
  if (PACKED) return w + (long long)(n / 16) * ksteps * (16 * Traits<FMT>::KSTEP) + 16 * lane;
  return w + (n + (lane & 15)) * ld + 16 * (lane >> 4);
}

// ---------------------------------------------------------------------- up --
// 16 columns of h: 16 gate and 16 up rows of one expert, K split over the
// waves, their sums joined through LDS in wave order.
struct UpLds {
  Choices c;
  v4i part[kWaves - 1][2][2][64];
};

template <int FMT, bool PACKED, int MB>
__device__ __forceinline__ void up_tile(const MoeLayerArgs& a, int n0, const Expert& x,
                                        UpLds& lds) {
  typedef typename Traits<FMT>::Frag Frag;
  typedef typename Traits<FMT>::Acc Acc;
  constexpr int KSTEP = Traits<FMT>::KSTEP;
  constexpr bool BLOCK = FMT == BLOCK_FP8;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int ksteps = (a.D + KSTEP - 1) / KSTEP, kfull = a.D / KSTEP, G = a.D / kGroup;
  const uint8_t* w1 = a.w1 + x.e * a.w1_stride;
  const float* s1 = a.s1 + x.e * a.s1_stride;
  const uint8_t* wp[2] = {weight_rows<FMT, PACKED>(w1, a.ldw1, ksteps, n0),
                          weight_rows<FMT, PACKED>(w1, a.ldw1, ksteps, a.I + n0)};
  const uint8_t* xp[MB];
  const float* sxp[MB];
  int entry[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    entry[b] = lds.c.entry[min(16 * b + r, x.tokens - 1)];
    const int t = entry[b] / a.topk;
    xp[b] = a.xq + t * a.ldq + 16 * g;
    sxp[b] = a.sx + (BLOCK ? (long long)t * G : t);
  }
  const float* swp[2] = {s1 + (BLOCK ? (long long)(n0 / kGroup) * G : n0 + 4 * g),
                         s1 + (BLOCK ? (long long)((a.I + n0) / kGroup) * G : a.I + n0 + 4 * g)};
  Acc acc[MB][2];
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[b][j] = Acc{0, 0, 0, 0};
  products<FMT, 2, MB, FMT == W8A8_INT8 ? 4 : 2>(
      acc, ksteps * wave / kWaves, ksteps * (wave + 1) / kWaves, kfull,
      [&](int j, int k) -> Frag {
        if constexpr (PACKED)
          return load_packed<FMT>(wp[j], k);
        else
          return load_frag<FMT>(wp[j], k);
      },
      [&](int b, int k) -> Frag { return load_frag<FMT>(xp[b], k); },
      [&](int j, int b, int k) { return sxp[b][k] * swp[j][k]; },
      [&](int j) -> Frag {
        if constexpr (PACKED)
          return load_packed<FMT>(wp[j], kfull);
        else
          return load_frag_tail<FMT>(wp[j], kfull, 16 * g, a.D);
      },
      [&](int b) -> Frag { return load_frag_tail<FMT>(xp[b], kfull, 16 * g, a.D); });
  // the waves' sums
  if (wave > 0) {
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j) lds.part[wave - 1][b][j][lane] = __builtin_bit_cast(v4i, acc[b][j]);
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int w = 0; w < kWaves - 1; ++w)
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[b][j] += __builtin_bit_cast(Acc, lds.part[w][b][j][lane]);
  // lane (r, g): token r of block b, columns n0 + 4 g .. + 3
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    v4f h;
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float gate, up;
      if constexpr (BLOCK) {
        gate = acc[b][0][i];
        up = acc[b][1][i];
      } else {
        gate = (float)acc[b][0][i] * sxp[b][0] * swp[0][i];
        up = (float)acc[b][1][i] * sxp[b][0] * swp[1][i];
      }
      h[i] = silu(gate) * up;
      top = max(top, abs_bits(h[i]));
    }
    top = max(top, (unsigned)__shfl_xor((int)top, 16, 64));
    top = max(top, (unsigned)__shfl_xor((int)top, 32, 64));
    if (16 * b + r < x.tokens) {
      *reinterpret_cast<v4f*>(a.h + (long long)entry[b] * a.I + n0 + 4 * g) = h;
      if (g == 0) a.hmax[(long long)entry[b] * (a.I / 16) + n0 / 16] = __uint_as_float(top);
    }
  }
}

template <int FMT, bool PACKED>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(MoeLayerArgs a) {
  __shared__ UpLds lds;
  const Expert x = find_expert(a, blockIdx.y, lds.c);
  if (x.e < 0) return;
  if (x.tokens <= 16)
    up_tile<FMT, PACKED, 1>(a, blockIdx.x * 16, x, lds);
  else
    up_tile<FMT, PACKED, 2>(a, blockIdx.x * 16, x, lds);
}

// -------------------------------------------------------------------- down --
// 64 columns of y for one expert: each wave 16 of its weight rows over the
// whole of I, the tokens' codes from LDS, where the workgroup makes them from h
// `chunk` columns at a time.
constexpr int kColumns = 16 * kWaves;
constexpr int kPad = 16;  // bytes that move a row's codes on by four LDS banks

extern __shared__ __align__(16) uint8_t codes[];

struct DownLds {
  Choices c;
  float scale[kLayerTokens];  // (one scale a token)
  int last;
};

template <int FMT, bool PACKED, int MB>
__device__ __forceinline__ void down_tile(const MoeLayerArgs& a, int n0, const Expert& x,
                                          DownLds& lds) {
  typedef typename Traits<FMT>::Frag Frag;
  typedef typename Traits<FMT>::Acc Acc;
  constexpr int KSTEP = Traits<FMT>::KSTEP;
  constexpr bool BLOCK = FMT == BLOCK_FP8, INT8 = FMT == W8A8_INT8;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int ksteps = (a.I + KSTEP - 1) / KSTEP, G = a.I / kGroup;
  const uint8_t* w2 = a.w2 + x.e * a.w2_stride;
  const float* s2 = a.s2 + x.e * a.s2_stride;
  // (waves past the last column repeat the last whole block, and store nothing)
  const int n = min(n0 + 16 * wave, a.D - 16);
  const uint8_t* wp = weight_rows<FMT, PACKED>(w2, a.ldw2, ksteps, n);
  const int stride = a.chunk + kPad;
  float* gscale = reinterpret_cast<float*>(codes + (long long)x.tokens * stride);  // Block_FP8's

  if constexpr (!BLOCK) {  // a token's scale: its waves' maxima
    for (int t = wave; t < x.tokens; t += kWaves) {
      const float* m = a.hmax + (long long)lds.c.entry[t] * (a.I / 16);
      unsigned top = 0;
      for (int i = lane; i < a.I / 16; i += 64) top = max(top, __float_as_uint(m[i]));
      top = wave_umax(top);
      if (lane == 0) lds.scale[t] = act_scale<INT8>(__uint_as_float(top));
    }
    __syncthreads();
  }
  Acc acc[MB][1];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b][0] = Acc{0, 0, 0, 0};
  for (int c0 = 0; c0 < a.I; c0 += a.chunk) {
    const int cols = min(a.chunk, a.I - c0), per = (cols + kGroup - 1) / kGroup * (kGroup / 8);
    if (c0) __syncthreads();  // the last chunk's codes have been read
    // eight columns a thread; zeros up to a whole step
    for (int i = threadIdx.x; i < x.tokens * per; i += kThreads) {
      const int t = i / per, k = 8 * (i - t * per);
      v2u q = {0u, 0u};
      if (k < cols) {
        const float* h = a.h + (long long)lds.c.entry[t] * a.I + c0 + k;
        float f[8];
        __builtin_memcpy(f, h, 32);
        float s;
        if constexpr (BLOCK) {
          const float* m = a.hmax + (long long)lds.c.entry[t] * (a.I / 16) + (c0 + k) / kGroup * 8;
          unsigned top = 0;
#pragma unroll
          for (int u = 0; u < 8; ++u) top = max(top, __float_as_uint(m[u]));
          s = act_scale<false>(__uint_as_float(top));
          if (k % kGroup == 0) gscale[t * (a.chunk / kGroup) + k / kGroup] = s;
        } else {
          s = lds.scale[t];
        }
        q = encode_values<INT8>(f, s, act_recip(s));
      }
      *reinterpret_cast<v2u*>(codes + t * stride + k) = q;
    }
    __syncthreads();
    const uint8_t* xp[MB];
    const float* sxp[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      const int t = min(16 * b + r, x.tokens - 1);
      xp[b] = codes + t * stride + 16 * g;
      sxp[b] = gscale + t * (a.chunk / kGroup);
    }
    const float* swp = s2 + (long long)(n / kGroup) * G;
    const int kb = c0 / KSTEP;
    auto tokens = [&](int b, int k) -> Frag { return load_frag<FMT>(xp[b], k - kb); };
    products<FMT, 1, MB, INT8 ? 4 : 2>(
        acc, kb, (c0 + cols + KSTEP - 1) / KSTEP, a.I / KSTEP,
        [&](int, int k) -> Frag {
          if constexpr (PACKED)
            return load_packed<FMT>(wp, k);
          else
            return load_frag<FMT>(wp, k);
        },
        tokens, [&](int, int b, int k) { return sxp[b][k - kb] * swp[k]; },
        [&](int) -> Frag {
          if constexpr (PACKED)
            return load_packed<FMT>(wp, a.I / KSTEP);
          else
            return load_frag_tail<FMT>(wp, a.I / KSTEP, 16 * g, a.I);
        },
        [&](int b) -> Frag { return tokens(b, a.I / KSTEP); });
  }
  // The experts' outputs, lane (r, g): token r of block b, columns n + 4 g .. +
  // 3; written through to where the last workgroup reads them, acknowledged
  // before this one counts itself in (the split-K hand-off of the small-M GEMM).
  const __amdgpu_buffer_rsrc_t out = coherent_rsrc(a.part, a.T * a.topk * a.D * 4);
  if (n0 + 16 * wave < a.D) {
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      const int t = 16 * b + r;
      v4f p;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (BLOCK)
          p[i] = acc[b][0][i];
        else
          p[i] = (float)acc[b][0][i] * lds.scale[min(t, x.tokens - 1)] * s2[n + 4 * g + i];
      }
      if (t < x.tokens)
        coherent_store16(out, (lds.c.entry[t] * a.D + n + 4 * g) * 4, __builtin_bit_cast(v4i, p));
    }
  }
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __syncthreads();
  if (threadIdx.x == 0) {
    // (the third word of a tile's counter line: it counts from zero, and the
    // last workgroup clears it)
    unsigned* counter = a.counters + (long long)blockIdx.x * kCounterWords + 2;
    const unsigned before =
        __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    lds.last = before == (unsigned)x.active - 1;
    if (lds.last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

template <int FMT, bool PACKED>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeLayerArgs a) {
  __shared__ DownLds lds;
  const Expert x = find_expert(a, blockIdx.y, lds.c);
  const int n0 = blockIdx.x * kColumns;
  if (x.e < 0) {
    if (x.active || blockIdx.y) return;  // (no token has an expert: zeros)
  } else {
    if (x.tokens <= 16)
      down_tile<FMT, PACKED, 1>(a, n0, x, lds);
    else
      down_tile<FMT, PACKED, 2>(a, n0, x, lds);
    if (!lds.last) return;
  }
  // y of the tile's columns, four a thread, in the order of the choices
  const __amdgpu_buffer_rsrc_t part = coherent_rsrc(a.part, a.T * a.topk * a.D * 4);
  constexpr int kBatch = 8;
  for (int i = threadIdx.x; i < a.T * (kColumns / 4); i += kThreads) {
    const int t = i / (kColumns / 4), n = n0 + 4 * (i % (kColumns / 4));
    if (n >= a.D) continue;
    v4f sum = {0, 0, 0, 0};
    for (int j0 = 0; j0 < a.topk; j0 += kBatch) {
      v4i v[kBatch];
      float w[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int at = t * a.topk + j0 + j;
        const bool on = j0 + j < a.topk && lds.c.ids[at] >= 0;
        v[j] = v4i{0, 0, 0, 0};
        w[j] = 0.0f;
        if (on) {
          v[j] = coherent_load16(part, (served_by(lds.c, at, t, a.topk) * a.D + n) * 4);
          w[j] = a.weights[at];
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const v4f p = __builtin_bit_cast(v4f, v[j]);
#pragma unroll
        for (int u = 0; u < 4; ++u) sum[u] = __builtin_fmaf(w[j], p[u], sum[u]);
      }
    }
    uint16_t* y = a.y + t * a.ldy + n;
#pragma unroll
    for (int u = 0; u < 4; ++u) y[u] = (uint16_t)bf16_bits(sum[u]);
  }
}

template <int FMT, bool PACKED>
hipError_t launch_up(const MoeLayerArgs& a, int slots, hipStream_t s) {
  return launch_kernel(moe_up_kernel<FMT, PACKED>, dim3((unsigned)(a.I / 16), (unsigned)slots),
                       dim3(kThreads), 0, s, a);
}
template <int FMT, bool PACKED>
hipError_t launch_down(const MoeLayerArgs& a, int slots, hipStream_t s) {
  const size_t lds = (size_t)a.T * (a.chunk + kPad + (FMT == BLOCK_FP8 ? a.chunk / kGroup * 4 : 0));
  return launch_kernel(moe_down_kernel<FMT, PACKED>,
                       dim3((unsigned)((a.D + kColumns - 1) / kColumns), (unsigned)slots),
                       dim3(kThreads), lds, s, a);
}
template <int FMT>
hipError_t launch_layer(bool packed1, bool packed2, const MoeLayerArgs& a, hipStream_t s) {
  const int slots = a.E < a.T * a.topk ? a.E : a.T * a.topk;
  const hipError_t e =
      packed1 ? launch_up<FMT, true>(a, slots, s) : launch_up<FMT, false>(a, slots, s);
  if (e != hipSuccess) return e;
  return packed2 ? launch_down<FMT, true>(a, slots, s) : launch_down<FMT, false>(a, slots, s);
}

}  // namespace

hipError_t launch_moe_layer(int fmt, bool packed1, bool packed2, const MoeLayerArgs& a,
                            hipStream_t s) {
  switch (fmt) {
    case FP8_DYNAMIC: return launch_layer<FP8_DYNAMIC>(packed1, packed2, a, s);
    case W8A8_INT8: return launch_layer<W8A8_INT8>(packed1, packed2, a, s);
    case BLOCK_FP8: return launch_layer<BLOCK_FP8>(packed1, packed2, a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace w8
