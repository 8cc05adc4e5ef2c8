// The experts of a few tokens as a whole, in two launches or three:
//
//   up    a = x W1_e^T for the tokens of expert e, gate and up halves;
//         h = silu(a_gate) a_up in fp32
//         (codes of h in the format, where many tiles would make them again)
//   down  hq = codes of h in the format; p = hq W2_e^T;
//         y[t] = base[t] + sum_j weights[t, j] p[t, j], by the last workgroup of
//         a column tile to arrive
//
// The weights' bytes are nearly all that a launch moves, so every workgroup
// streams its own piece of one expert's weights into MFMA registers, as the
// small-M GEMM does (A = weights, B = tokens: a lane's accumulators belong to
// one token).  Which experts have tokens, and which tokens, every workgroup
// finds for itself from the T x topk choices, so a launch needs no lists and
// reads no weights of an expert without tokens.
//
// Measured with 128 experts, top 8, of 2048 x 768, row-major (a call among others,
// and the kernels' medians in a trace, where they do not overlap; the weights of the
// experts that are chosen, and their rate): 1 token in Block_FP8 14.4 us (38 MB: up
// 8.8, down 7.4, two chains of choices, weights and sums that few workgroups run
// once); 8 tokens in int8 53.6 us (244 MB; up 36.8, 4.4 TB/s, down 24.4, 3.3); 32
// tokens in fp8 97.9 us (527 MB; up 67.9, 5.2 TB/s, down 42.8, 4.1), by the weights'
// bytes.  Of down's time 3.5 to 5 us are the hand-off of the outputs to the workgroup
// that sums them, about what a launch of its own would take for that.
#include <type_traits>

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
  int ids[kMaxEntries];                  // (-1: no expert of this call's)
  unsigned set[kMaxExperts / 32];        // experts with tokens
  int entry[kWaves][kLayerTokens];       // first entry of each of the expert's tokens
};
struct Expert {
  int e;       // -1: none for this workgroup
  int tokens;  // of the expert
};

// Lane t's first entry with the expert (-1: none) becomes the wave's list.
__device__ __forceinline__ int list_tokens(int first, Choices& c) {
  const int lane = threadIdx.x & 63;
  const unsigned long long mine = __ballot(first >= 0);
  if (first >= 0) c.entry[threadIdx.x >> 6][__popcll(mine & ((1ull << lane) - 1))] = first;
  // (the wave's own LDS, which it accesses in order; reads of the list, which lanes
  // write for each other, stay behind the write.  A fence of all memory here, which
  // holds the first weights' addresses back too, costs up to 2%.)
  __builtin_amdgcn_wave_barrier();
  return __popcll(mine);
}

// The expert of a launch's slot; every wave finds it for itself.
//
// Up to 64 entries, no more than experts: slot s is entry s, if it is the first
// of its expert.  The entries lie in the lanes, and nothing waits for another
// wave.
__device__ __forceinline__ Expert find_among_few(const MoeLayerArgs& a, int slot, Choices& c) {
  const int lane = threadIdx.x & 63, n = a.T * a.topk;
  const int id = lane < n ? a.experts[lane] : -1;
  const int e = __builtin_amdgcn_readlane(id, slot);
  const unsigned long long same = __ballot(lane < n && id == e);
  if ((unsigned)e >= (unsigned)a.E || __builtin_ctzll(same) != slot) return {-1, 0};
  const unsigned long long mine =
      lane < a.T ? same >> (lane * a.topk) & ((1ull << (a.topk - 1) << 1) - 1) : 0;
  return {e, list_tokens(mine ? lane * a.topk + __builtin_ctzll(mine) : -1, c)};
}

// Otherwise slot s is the s-th of the experts that have tokens, from a set of
// them in LDS (*active: how many there are).
__device__ __forceinline__ void load_choices(const MoeLayerArgs& a, Choices& c) {
  if (threadIdx.x < kMaxExperts / 32) c.set[threadIdx.x] = 0u;
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * a.topk; i += kThreads) {
    const int id = a.experts[i];
    const bool on = (unsigned)id < (unsigned)a.E;
    c.ids[i] = on ? id : -1;
    if (on) atomicOr(&c.set[id >> 5], 1u << (id & 31));
  }
  __syncthreads();
}
__device__ __forceinline__ int count_active(const Choices& c) {
  const int lane = threadIdx.x & 63;
  return __builtin_amdgcn_readlane(
      wave_scan(lane < kMaxExperts / 32 ? __popc(c.set[lane]) : 0), 63);
}
__device__ __forceinline__ Expert find_among_all(const MoeLayerArgs& a, int slot, Choices& c) {
  const int lane = threadIdx.x & 63;
  load_choices(a, c);
  const unsigned word = lane < kMaxExperts / 32 ? c.set[lane] : 0u;
  const int upto = wave_scan(__popc(word));
  const unsigned long long past = __ballot(upto > slot);
  if (!past) return {-1, 0};
  const int l = __builtin_ctzll(past);
  unsigned bits = __builtin_amdgcn_readlane((int)word, l);
  for (int i = l ? __builtin_amdgcn_readlane(upto, l - 1) : 0; i < slot; ++i) bits &= bits - 1;
  const int e = 32 * l + __builtin_ctz(bits);
  int first = -1;
  if (lane < a.T)
    for (int j = a.topk - 1; j >= 0; --j)
      if (c.ids[lane * a.topk + j] == e) first = lane * a.topk + j;
  return {e, list_tokens(first, c)};
}
__device__ __forceinline__ Expert find_expert(const MoeLayerArgs& a, int slot, Choices& c) {
  return a.few ? find_among_few(a, slot, c) : find_among_all(a, slot, c);
}

// ids becomes, for every entry, the one whose outputs serve it: the first of its
// token with the same expert (-1: none).
__device__ __forceinline__ void find_outputs(const MoeLayerArgs& a, Choices& c) {
  const int n = a.T * a.topk;
  int at[kMaxEntries / kThreads];
#pragma unroll
  for (int q = 0; q < kMaxEntries / kThreads; ++q) {
    const int i = threadIdx.x + q * kThreads;
    at[q] = -1;
    if (i < n && c.ids[i] >= 0) {
      at[q] = i / a.topk * a.topk;
      while (c.ids[at[q]] != c.ids[i]) ++at[q];
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kMaxEntries / kThreads; ++q)
    if ((int)threadIdx.x + q * kThreads < n) c.ids[threadIdx.x + q * kThreads] = at[q];
  __syncthreads();
}

// The products of NB blocks of 16 weight rows with MB blocks of 16 token rows
// over the whole K-steps [la, lfull).  weights(j, k) and tokens(b, k) are the
// operands of step k, wscale(j, k) and xscale(b, k) Block_FP8's factors.  R
// steps are in flight: begin() issues the first R, run() multiplies each and
// issues the one R steps on into the same registers.  (Loads past the last step
// repeat it.)  EARLY: tokens come from memory, with the weights; else from LDS,
// when they are multiplied.
template <int FMT, int NB, int MB, int R, bool EARLY, class W, class X, class WS, class XS>
struct Products {
  typedef typename Traits<FMT>::Frag Frag;
  typedef typename Traits<FMT>::Acc Acc;
  static constexpr bool BLOCK = FMT == BLOCK_FP8;
  W weights;
  X tokens;
  WS wscale;
  XS xscale;
  int la, lfull;
  Frag w[R][NB], x[EARLY ? R : 1][MB];
  float ws[BLOCK ? R : 1][NB], xs[BLOCK && EARLY ? R : 1][MB];

  __device__ __forceinline__ Products(int la, int lfull, W w, X x, WS ws, XS xs)
      : weights(w), tokens(x), wscale(ws), xscale(xs), la(la), lfull(lfull) {}
  __device__ __forceinline__ void load(int u, int step) {
    const int k = min(step, lfull - 1);
#pragma unroll
    for (int j = 0; j < NB; ++j) w[u][j] = weights(j, k);
    if constexpr (BLOCK) {
#pragma unroll
      for (int j = 0; j < NB; ++j) ws[u][j] = wscale(j, k);
    }
    if constexpr (EARLY) {
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        x[u][b] = tokens(b, k);
        if constexpr (BLOCK) xs[u][b] = xscale(b, k);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  // FP8_Dynamic's running sum stays in the instruction's accumulator, which keeps it
  // as exactly as an fp32 sum of the steps would (codes of normal values, 1 to 128
  // steps: 1.4e-5 to 1.55e-5 of the result in the root mean square either way).  That
  // error is the instruction's rounding of a step's products among each other, and
  // the forms of 32 codes an instruction have the same.
  static __device__ __forceinline__ void multiply(Acc& c, const Frag& w, const Frag& x, float sc) {
    if constexpr (BLOCK) {
      const Acc p = mma<FMT, 1>(w, x, Acc{0, 0, 0, 0});
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = __builtin_fmaf(p[i], sc, c[i]);
    } else {
      c = mma<FMT, 1>(w, x, c);
    }
  }
  __device__ __forceinline__ void use(int u, int k, Acc (&acc)[MB][NB]) {
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      Frag xf;
      float sc = 0.0f;
      if constexpr (EARLY) {
        xf = x[u][b];
        if constexpr (BLOCK) sc = xs[u][b];
      } else {
        xf = tokens(b, k);
        if constexpr (BLOCK) sc = xscale(b, k);
      }
#pragma unroll
      for (int j = 0; j < NB; ++j)
        multiply(acc[b][j], w[u][j], xf, BLOCK ? sc * ws[u][j] : 0.0f);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  __device__ __forceinline__ void begin() {
    if (la >= lfull) return;
#pragma unroll
    for (int u = 0; u < R; ++u) load(u, la + u);
  }
  __device__ __forceinline__ void run(Acc (&acc)[MB][NB]) {
    int k = la;
    for (; k + R < lfull; k += R) {
#pragma unroll
      for (int u = 0; u < R; ++u) {
        use(u, k + u, acc);
        load(u, k + R + u);
      }
    }
#pragma unroll
    for (int u = 0; u < R; ++u)
      if (k + u < lfull) use(u, k + u, acc);
  }
};
template <int FMT, int NB, int MB, int R, bool EARLY, class W, class X, class WS, class XS>
__device__ __forceinline__ Products<FMT, NB, MB, R, EARLY, W, X, WS, XS> products(
    int la, int lfull, W w, X x, WS ws, XS xs) {
  return {la, lfull, w, x, ws, xs};
}

// Steps in flight: so many 128-byte pieces of a weight row's K.
template <int FMT>
constexpr int steps(int pieces) {
  return FMT == W8A8_INT8 ? 2 * pieces : pieces;
}

// The wave's first fragment (PACKED) or row of 16 weight rows from row n.
template <int FMT, bool PACKED>
__device__ __forceinline__ const uint8_t* weight_rows(const uint8_t* w, long long ld, int ksteps,
                                                      int n) {
  const int lane = threadIdx.x & 63;
  if (PACKED) return w + (long long)(n / 16) * ksteps * (16 * Traits<FMT>::KSTEP) + 16 * lane;
  return w + (n + (lane & 15)) * ld + 16 * (lane >> 4);
}
template <int FMT, bool PACKED>
__device__ __forceinline__ typename Traits<FMT>::Frag weight_step(const uint8_t* w, int k) {
  if constexpr (PACKED)
    return load_packed<FMT>(w, k);
  else
    return load_frag<FMT>(w, k);
}
// Where K ends inside step k: zeros past it (packed weights hold them).
template <int FMT, bool PACKED>
__device__ __forceinline__ typename Traits<FMT>::Frag weight_tail(const uint8_t* w, int k, int K) {
  if constexpr (PACKED)
    return load_packed<FMT>(w, k);
  else
    return load_frag_tail<FMT>(w, k, 16 * ((threadIdx.x & 63) >> 4), K);
}
// One value for the whole wave: a scalar load, off the vector-memory path.
__device__ __forceinline__ float uniform_load(const float* p) {
  return *(const __attribute__((address_space(4))) float*)p;
}

// ---------------------------------------------------------------------- up --
// 16 columns of h: 16 gate and 16 up rows of one expert, K split over the
// waves, their sums joined through LDS in wave order.  So 128 bytes of 64 rows a
// step are in flight a workgroup, two steps deep, and five workgroups or six (72 to
// 86 registers) share a compute unit, four (97 to 110) where experts may have more
// than 16 tokens (calls of 8 tokens in int8 as above, one to four steps deep: 64.5,
// 62.8, 69.3 and 62.7 us; 1 token 14.5, 14.7, 16.6 and 14.9; 32 tokens in fp8 105.5,
// 105.4, 118.8 and 116.7, where registers leave room for three workgroups and two).
constexpr int kUpPieces = 2;

template <int MB, int KW>
struct UpLds {
  Choices c;
  v4i part[KW > 1 ? (KW - 1) * MB * 2 : 1][64];
};

// MB blocks of 16 tokens, all that the expert has; KW waves share a block of
// columns, wave kw a part of its K.
template <int FMT, bool PACKED, int MB, int KW>
__device__ __forceinline__ void up_tile(const MoeLayerArgs& a, int n0, const Expert& x,
                                        const Choices& c, v4i (*part)[64]) {
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
    entry[b] = c.entry[wave][min(16 * b + r, x.tokens - 1)];
    const int t = entry[b] / a.topk;
    xp[b] = a.xq + t * a.ldq + 16 * g;
    sxp[b] = a.sx + (BLOCK ? (long long)t * G : t);
  }
  const float* swp[2] = {s1 + (BLOCK ? (long long)(n0 / kGroup) * G : n0),
                         s1 + (BLOCK ? (long long)((a.I + n0) / kGroup) * G : a.I + n0)};
  Acc acc[MB][2];
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[b][j] = Acc{0, 0, 0, 0};
  const int kw = KW > 1 ? wave : 0;
  const int la = ksteps * kw / KW, lb = ksteps * (kw + 1) / KW;
  auto p = products<FMT, 2, MB, steps<FMT>(kUpPieces), true>(
      la, min(lb, kfull), [&](int j, int k) -> Frag { return weight_step<FMT, PACKED>(wp[j], k); },
      [&](int b, int k) -> Frag { return load_frag<FMT>(xp[b], k); },
      [&](int j, int k) { return uniform_load(swp[j] + k); },
      [&](int b, int k) { return sxp[b][k]; });
  p.begin();
  // the epilogue's scales, behind the first weights
  float sx[MB], sw[2][4];
  if constexpr (!BLOCK) {
    if (kw == 0) {
#pragma unroll
      for (int b = 0; b < MB; ++b) sx[b] = *sxp[b];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) sw[j][i] = swp[j][4 * g + i];
    }
  }
  p.run(acc);
  if constexpr (!BLOCK) {  // (Block_FP8's K is whole steps)
    if (lb > kfull && la < lb) {
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const Frag t = load_frag_tail<FMT>(xp[b], kfull, 16 * g, a.D);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          p.multiply(acc[b][j], weight_tail<FMT, PACKED>(wp[j], kfull, a.D), t, 0.0f);
      }
    }
  }
  // the waves' sums
  if constexpr (KW > 1) {
    if (kw > 0) {
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          part[((kw - 1) * MB + b) * 2 + j][lane] = __builtin_bit_cast(v4i, acc[b][j]);
    }
    __syncthreads();
  }
  if (kw == 0) {
#pragma unroll
    for (int w = 0; w < KW - 1; ++w)
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[b][j] += __builtin_bit_cast(Acc, part[(w * MB + b) * 2 + j][lane]);
    // lane (r, g): token r of block b, columns n0 + 4 g .. + 3
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      v4f h;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float gate = (float)acc[b][0][i], up = (float)acc[b][1][i];
        if constexpr (!BLOCK) {
          gate *= sx[b] * sw[0][i];
          up *= sx[b] * sw[1][i];
        }
        h[i] = silu(gate) * up;
      }
      if (16 * b + r < x.tokens)
        *reinterpret_cast<v4f*>(a.h + (long long)entry[b] * a.I + n0 + 4 * g) = h;
    }
  }
}

template <int FMT, bool PACKED, int MB, int KW>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(MoeLayerArgs a) {
  __shared__ UpLds<MB, KW> lds;
  const Expert x = find_expert(a, blockIdx.y, lds.c);
  if (x.e < 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = KW > 1 ? blockIdx.x * 16 : (blockIdx.x * kWaves + wave) * 16;
  if (n0 >= a.I) return;  // (a wave by itself, KW == 1)
  if (MB == 1 || x.tokens <= 16)
    up_tile<FMT, PACKED, 1, KW>(a, n0, x, lds.c, lds.part);
  else
    up_tile<FMT, PACKED, MB, KW>(a, n0, x, lds.c, lds.part);
}

// -------------------------------------------------------------------- down --
// 64 columns of y for one expert: each wave 16 of its weight rows over the whole
// of I, the tokens' codes from LDS, where the workgroup makes them from h
// `chunk` columns at a time, or from memory, if they are there.  Two steps are in
// flight (calls as above, two, three, four and six: 8 tokens 62.8, 62.9, 64.3 and 62.8
// us, 32 tokens 105.4, 105.8, 110.4 and 106.8).
constexpr int kColumns = 16 * kWaves;
constexpr int kPad = 16;  // bytes that move a row's codes on by four LDS banks

extern __shared__ __align__(16) uint8_t codes[];

struct DownLds {
  Choices c;
  unsigned top[kLayerTokens];  // (one scale a token) the bits of the largest |h|
  int last;
};

// Eight of the expert's hidden values: those of thread i of a chunk's
// `per` threads a token, from column c0 on; zeros past column `cols`.
struct Hidden {
  float f[8];
};
__device__ __forceinline__ Hidden load_hidden(const MoeLayerArgs& a, const int* entry, int i,
                                              int per, int c0, int cols) {
  Hidden v = {};
  const int t = i / per, k = 8 * (i - t * per);
  if (k < cols) __builtin_memcpy(v.f, a.h + (long long)entry[t] * a.I + c0 + k, 32);
  return v;
}
// Two of them a thread, from piece i0 on of `count`; their loads are all in
// flight.
constexpr int kHeld = 2;
__device__ __forceinline__ void load_hidden(const MoeLayerArgs& a, const int* entry, int i0,
                                            int count, int per, int c0, int cols,
                                            Hidden (&v)[kHeld]) {
#pragma unroll
  for (int q = 0; q < kHeld; ++q) {
    const int i = i0 + (int)threadIdx.x + q * kThreads;
    v[q] = Hidden{};
    if (i < count) v[q] = load_hidden(a, entry, i, per, c0, cols);
  }
}
__device__ __forceinline__ unsigned largest(const Hidden& v) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v.f[i]));
  return m;
}

// CODED: moe_encode_kernel has made the tokens' codes.
template <int FMT, bool PACKED, int MB, bool CODED>
__device__ __forceinline__ void down_tile(const MoeLayerArgs& a, int n0, const Expert& x,
                                          DownLds& lds) {
  typedef typename Traits<FMT>::Frag Frag;
  typedef typename Traits<FMT>::Acc Acc;
  constexpr int KSTEP = Traits<FMT>::KSTEP;
  constexpr bool BLOCK = FMT == BLOCK_FP8, INT8 = FMT == W8A8_INT8;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int ksteps = (a.I + KSTEP - 1) / KSTEP, kfull = a.I / KSTEP, G = a.I / kGroup;
  const uint8_t* w2 = a.w2 + x.e * a.w2_stride;
  const float* s2 = a.s2 + x.e * a.s2_stride;
  // (waves past the last column repeat the last whole block, and store nothing)
  const int n = min(n0 + 16 * wave, a.D - 16);
  const uint8_t* wp = weight_rows<FMT, PACKED>(w2, a.ldw2, ksteps, n);
  const float* swp = s2 + (BLOCK ? (long long)(n / kGroup) * G : n + 4 * g);
  const int* entry = lds.c.entry[wave];
  const int stride = a.chunk + kPad;
  float* gscale = reinterpret_cast<float*>(codes + (long long)x.tokens * stride);  // Block_FP8's

  // the workgroup's columns of I, in whole 128s
  const int groups = (a.I + kGroup - 1) / kGroup;
  const int lo = groups * (int)blockIdx.z / a.splits * kGroup;
  const int hi = min(groups * ((int)blockIdx.z + 1) / a.splits * kGroup, a.I);

  const uint8_t* xp[MB];
  const float* sxp[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int t = min(16 * b + r, x.tokens - 1);
    xp[b] = codes + t * stride + 16 * g;
    sxp[b] = gscale + t * (a.chunk / kGroup);
  }
  Acc acc[MB][1];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b][0] = Acc{0, 0, 0, 0};
  float sw[4];
  if constexpr (CODED) {
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      const int e = entry[min(16 * b + r, x.tokens - 1)];
      xp[b] = a.hq + (long long)e * a.ldh + 16 * g;
      sxp[b] = a.hs + (BLOCK ? (long long)e * G : e);
    }
    const int la = lo / KSTEP, lb = (hi + KSTEP - 1) / KSTEP;
    auto p = products<FMT, 1, MB, steps<FMT>(2), true>(
        la, min(lb, kfull), [&](int, int k) -> Frag { return weight_step<FMT, PACKED>(wp, k); },
        [&](int b, int k) -> Frag { return load_frag<FMT>(xp[b], k); },
        [&](int, int k) { return uniform_load(swp + k); },
        [&](int b, int k) { return sxp[b][k]; });
    p.begin();
    if constexpr (!BLOCK) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sw[i] = swp[i];
    }
    p.run(acc);
    if constexpr (!BLOCK) {
      if (lb > kfull) {
        const Frag w = weight_tail<FMT, PACKED>(wp, kfull, a.I);
#pragma unroll
        for (int b = 0; b < MB; ++b)
          p.multiply(acc[b][0], w, load_frag_tail<FMT>(xp[b], kfull, 16 * g, a.I), 0.0f);
      }
    }
  }
  for (int c0 = lo; !CODED && c0 < hi; c0 += a.chunk) {
    const int cols = min(a.chunk, hi - c0), per = (cols + kGroup - 1) / kGroup * (kGroup / 8);
    const int kb = c0 / KSTEP, kend = (c0 + cols + KSTEP - 1) / KSTEP;
    // a thread's first hidden values, then the first weights: loads return in
    // order, so that the codes are made while the weights arrive
    const int pieces = x.tokens * per;
    Hidden held[kHeld];
    load_hidden(a, entry, 0, pieces, per, c0, cols, held);
    auto p = products<FMT, 1, MB, steps<FMT>(2), false>(
        kb, min(kend, kfull), [&](int, int k) -> Frag { return weight_step<FMT, PACKED>(wp, k); },
        [&](int b, int k) -> Frag { return load_frag<FMT>(xp[b], k - kb); },
        [&](int, int k) { return uniform_load(swp + k); },
        [&](int b, int k) { return sxp[b][k - kb]; });
    p.begin();
    if constexpr (!BLOCK) {
      if (c0 == lo) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sw[i] = swp[i];
        // the tokens' largest values, over all of I
        if (threadIdx.x < kLayerTokens) lds.top[threadIdx.x] = 0u;
        __syncthreads();
        // (a token's threads are whole groups of 16 lanes)
        auto take = [&](int i0, int count, int each, const Hidden (&v)[kHeld]) {
#pragma unroll
          for (int q = 0; q < kHeld; ++q) {
            const int i = i0 + (int)threadIdx.x + q * kThreads;
            if (i >= count) continue;
            const unsigned m = seg16_umax(largest(v[q]));
            if ((i & 15) == 0) atomicMax(&lds.top[i / each], m);
          }
        };
        take(0, pieces, per, held);
        for (int c = 0; c < a.I; c += a.chunk) {
          const int more = min(a.chunk, a.I - c), each = (more + kGroup - 1) / kGroup * (kGroup / 8);
          // (those that are held are the first chunk's start, if I is not split)
          for (int i0 = c == 0 && a.splits == 1 ? kHeld * kThreads : 0; i0 < x.tokens * each; i0 += kHeld * kThreads) {
            Hidden v[kHeld];
            load_hidden(a, entry, i0, x.tokens * each, each, c, more, v);
            take(i0, x.tokens * each, each, v);
          }
        }
      }
    }
    __syncthreads();  // (and the last chunk's codes have been read)
    for (int i0 = 0; i0 < pieces; i0 += kHeld * kThreads) {
      if (i0) load_hidden(a, entry, i0, pieces, per, c0, cols, held);
#pragma unroll
      for (int q = 0; q < kHeld; ++q) {
        const int i = i0 + (int)threadIdx.x + q * kThreads;
        if (i >= pieces) continue;
        const int t = i / per, k = 8 * (i - t * per);
        float s;
        if constexpr (BLOCK) {  // 16 lanes hold a group
          s = act_scale<false>(__uint_as_float(seg16_umax(largest(held[q]))));
          if (k % kGroup == 0) gscale[t * (a.chunk / kGroup) + k / kGroup] = s;
        } else {
          s = act_scale<INT8>(__uint_as_float(lds.top[t]));
        }
        *reinterpret_cast<v2u*>(codes + t * stride + k) =
            encode_values<INT8>(held[q].f, s, act_recip(s));
      }
    }
    __syncthreads();
    p.run(acc);
    if constexpr (!BLOCK) {
      if (kend > kfull) {
        const Frag w = weight_tail<FMT, PACKED>(wp, kfull, a.I);
#pragma unroll
        for (int b = 0; b < MB; ++b)
          p.multiply(acc[b][0], w, load_frag<FMT>(xp[b], kfull - kb), 0.0f);
      }
    }
  }
  // The experts' outputs, lane (r, g): token r of block b, columns n + 4 g .. +
  // 3; written through to where the last workgroup reads them, acknowledged
  // before this one counts itself in (the split-K hand-off of the small-M GEMM).
  // int8's parts of I stay whole numbers, so that their sum is exact, and the
  // first part's workgroup leaves their scales behind the parts (whoever adds
  // them would read the experts' scales late).
  const bool whole = INT8 && a.splits > 1;
  const int n_entries = a.T * a.topk;
  const __amdgpu_buffer_rsrc_t out = coherent_rsrc(a.part, (a.splits + whole) * n_entries * a.D * 4);
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int t = 16 * b + r, at = min(t, x.tokens - 1);
    float sx = 0.0f;
    if constexpr (!BLOCK)
      sx = CODED ? a.hs[entry[at]] : act_scale<INT8>(__uint_as_float(lds.top[at]));
    v4f o, scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = (float)acc[b][0][i];
      if constexpr (!BLOCK) {
        scale[i] = sx * sw[i];
        o[i] *= scale[i];
      }
    }
    if (t >= x.tokens || n0 + 16 * wave >= a.D) continue;
    const int to = entry[at] * a.D + n + 4 * g;
    coherent_store16(out, ((int)blockIdx.z * n_entries * a.D + to) * 4,
                     whole ? __builtin_bit_cast(v4i, acc[b][0]) : __builtin_bit_cast(v4i, o));
    if (whole && blockIdx.z == 0)
      coherent_store16(out, (a.splits * n_entries * a.D + to) * 4, __builtin_bit_cast(v4i, scale));
  }
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  // (how many will, while the stores are on their way)
  if (a.few) load_choices(a, lds.c);
  const int active = count_active(lds.c) * a.splits;
  __builtin_amdgcn_s_waitcnt(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __syncthreads();
  if (threadIdx.x == 0) {
    // (the third word of a tile's counter line: it counts from zero, and the
    // last workgroup clears it)
    unsigned* counter = a.counters + (long long)blockIdx.x * kCounterWords + 2;
    const unsigned before =
        __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    lds.last = before == (unsigned)active - 1;
    if (lds.last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// y of a tile's columns, four a thread, in the order of the choices, an output's
// parts (SPLIT: of I; WHOLE: whole numbers, whose scales lie behind them) first; the
// loads of a batch are all in flight (left out: entry 0's, not used).
template <int BATCH, bool SPLIT, bool WHOLE>
__device__ __forceinline__ void sum_outputs(const MoeLayerArgs& a, int n0, const Choices& c) {
  const int n_entries = a.T * a.topk;
  const __amdgpu_buffer_rsrc_t part =
      coherent_rsrc(a.part, (a.splits + WHOLE) * n_entries * a.D * 4);
  for (int i = threadIdx.x; i < a.T * (kColumns / 4); i += kThreads) {
    const int t = i / (kColumns / 4), n = n0 + 4 * (i % (kColumns / 4));
    if (n >= a.D) continue;
    v4f sum = {0, 0, 0, 0};
    if (a.base) {
      uint16_t b[4];
      __builtin_memcpy(b, a.base + t * a.ldb + n, 8);
#pragma unroll
      for (int u = 0; u < 4; ++u) sum[u] = bf16_lo(b[u]);
    }
    for (int j0 = 0; j0 < a.topk; j0 += BATCH) {
      v4i v[BATCH];
      float w[BATCH];
      int from[BATCH];
      bool on[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        const int at = t * a.topk + min(j0 + j, a.topk - 1), id = c.ids[at];
        on[j] = j0 + j < a.topk && id >= 0;
        from[j] = max(id, 0);
        v[j] = coherent_load16(part, (from[j] * a.D + n) * 4);
        w[j] = a.weights[at];
      }
      typedef std::conditional_t<WHOLE, v4i, v4f> Part;
      Part q[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j) q[j] = __builtin_bit_cast(Part, v[j]);
      for (int z = 1; SPLIT && z < a.splits; ++z) {
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
          v[j] = coherent_load16(part, ((z * n_entries + from[j]) * a.D + n) * 4);
#pragma unroll
        for (int j = 0; j < BATCH; ++j) q[j] += __builtin_bit_cast(Part, v[j]);
      }
      // (loaded with the parts, the scales take registers of every second kernel in
      // int8: 8 tokens of 128 experts 61.3 us a call, so 60.5, calls in parts as fast)
      v4i scale[WHOLE ? BATCH : 1];
      if constexpr (WHOLE) {
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
          scale[j] = coherent_load16(part, ((a.splits * n_entries + from[j]) * a.D + n) * 4);
      }
      v4f p[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        if constexpr (WHOLE) {
          const v4f f = __builtin_bit_cast(v4f, scale[j]);
#pragma unroll
          for (int u = 0; u < 4; ++u) p[j][u] = (float)q[j][u] * f[u];
        } else {
          p[j] = q[j];
        }
      }
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          sum[u] = on[j] ? __builtin_fmaf(w[j], p[j][u], sum[u]) : sum[u];
      }
    }
    uint16_t y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) y[u] = (uint16_t)bf16_bits(sum[u]);
    __builtin_memcpy(a.y + t * a.ldy + n, y, 8);
  }
}

template <int FMT, bool PACKED, int MB, bool CODED>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeLayerArgs a) {
  __shared__ DownLds lds;
  const Expert x = find_expert(a, blockIdx.y, lds.c);
  const int n0 = blockIdx.x * kColumns;
  if (x.e < 0) {  // (no token has an expert: the base alone)
    if (blockIdx.y || blockIdx.z) return;
    if (a.few) load_choices(a, lds.c);
    if (count_active(lds.c)) return;
  } else {
    if (MB == 1 || x.tokens <= 16)
      down_tile<FMT, PACKED, 1, CODED>(a, n0, x, lds);
    else
      down_tile<FMT, PACKED, MB, CODED>(a, n0, x, lds);
    if (!lds.last) return;
  }
  find_outputs(a, lds.c);
  if (a.splits == 1)
    sum_outputs<8, false, false>(a, n0, lds.c);
  else
    sum_outputs<4, true, FMT == W8A8_INT8>(a, n0, lds.c);
}

// The codes and scales of an entry's hidden values, a workgroup each, with as many
// threads as take them at once (64 entries of 14336: 4.8 us, by 256 threads 9.0).
constexpr int kEncodeThreads = 1024;

template <int FMT>
__global__ __launch_bounds__(kEncodeThreads) void moe_encode_kernel(MoeLayerArgs a) {
  constexpr bool BLOCK = FMT == BLOCK_FP8, INT8 = FMT == W8A8_INT8;
  __shared__ unsigned tops[kEncodeThreads / 64];
  const int entry = blockIdx.x, id = a.experts[entry], threads = blockDim.x;
  // (of an expert that the token has chosen before nothing is there; nobody asks)
  if ((unsigned)id >= (unsigned)a.E) return;
  const int per = (a.I + kGroup - 1) / kGroup * (kGroup / 8);
  uint8_t* q = a.hq + (long long)entry * a.ldh;
  constexpr int N = 2;  // pieces of eight values in flight, the first two kept
  auto load = [&](int i0, Hidden (&v)[N]) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int i = i0 + (int)threadIdx.x + u * threads;
      v[u] = Hidden{};
      if (i < per) v[u] = load_hidden(a, &entry, i, per, 0, a.I);
    }
  };
  Hidden held[N];
  load(0, held);
  float s = 0.0f;
  if constexpr (!BLOCK) {
    unsigned top = 0;
#pragma unroll
    for (int u = 0; u < N; ++u) top = max(top, largest(held[u]));
    for (int i0 = N * threads; i0 < per; i0 += N * threads) {
      Hidden v[N];
      load(i0, v);
#pragma unroll
      for (int u = 0; u < N; ++u) top = max(top, largest(v[u]));
    }
    top = wave_umax(top);
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    for (int w = 0; w < threads / 64; ++w) top = max(top, tops[w]);
    s = act_scale<INT8>(__uint_as_float(top));
    if (threadIdx.x == 0) a.hs[entry] = s;
  }
  for (int i0 = 0; i0 < per; i0 += N * threads) {
    if (i0) load(i0, held);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int i = i0 + (int)threadIdx.x + u * threads;
      if (i >= per) continue;
      if constexpr (BLOCK) {  // 16 lanes hold a group
        s = act_scale<false>(__uint_as_float(seg16_umax(largest(held[u]))));
        if ((i & 15) == 0) a.hs[(long long)entry * (a.I / kGroup) + i / 16] = s;
      }
      if (8 * i < a.I)
        *reinterpret_cast<v2u*>(q + 8 * i) = encode_values<INT8>(held[u].f, s, act_recip(s));
    }
  }
}

// Few entries: 16 columns of y for all of them, one or several waves an entry
// (`parts`, a power of two, of I), so that their sum needs no hand-off between
// workgroups, which is what a call of so few bytes waits for (1 token, 8 experts
// of 2048 x 768: 6.6 us, 8.0 by the kernel above).
constexpr int kFewWaves = 16;

template <int FMT, bool PACKED>
__global__ __launch_bounds__(64 * kFewWaves) void moe_down_few_kernel(MoeLayerArgs a) {
  typedef typename Traits<FMT>::Frag Frag;
  typedef typename Traits<FMT>::Acc Acc;
  constexpr int KSTEP = Traits<FMT>::KSTEP;
  constexpr bool BLOCK = FMT == BLOCK_FP8, INT8 = FMT == W8A8_INT8;
  __shared__ decltype(Acc{}[0] + 0) sums[kFewWaves][16];  // by wave: the 16 columns
  __shared__ float outputs[kFewWaves][16];  // by entry
  __shared__ unsigned tops[kFewWaves];      // (one scale a token) the bits of the largest |h|
  __shared__ float scales[kFewWaves][16];   // by entry: of the 16 columns
  __shared__ float weights[kFewWaves];      // by entry
  __shared__ bool counts[kFewWaves];        // by entry: it is not left out
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int entry = wave >> __builtin_ctz(a.parts), part = wave & (a.parts - 1);
  const int g = lane >> 4, n = blockIdx.x * 16, entries = a.T * a.topk;
  const int id = lane < entries ? a.experts[lane] : -1;
  const int e = __builtin_amdgcn_readlane(id, entry);
  const bool on = (unsigned)e < (unsigned)a.E;
  // the hidden values of an expert that the token has chosen before are there
  const int first = entry / a.topk * a.topk;
  const int from = first + __builtin_ctzll(__ballot(lane < entries && id == e) >> first);
  const float weight = a.weights[entry];
  const int ksteps = (a.I + KSTEP - 1) / KSTEP, kfull = a.I / KSTEP, G = a.I / kGroup;
  const float* s2 = a.s2 + (on ? e * a.s2_stride : 0);
  const uint8_t* wp = weight_rows<FMT, PACKED>(a.w2 + (on ? e * a.w2_stride : 0), a.ldw2, ksteps, n);
  const float* swp = s2 + (BLOCK ? (long long)(n / kGroup) * G : n + 4 * g);
  // the wave's columns of I, in whole 128s
  const int groups = (a.I + kGroup - 1) / kGroup;
  const int lo = groups * part / a.parts * kGroup;
  const int hi = on ? min(groups * (part + 1) / a.parts * kGroup, a.I) : lo;
  const int stride = a.chunk + kPad;
  uint8_t* x = codes + wave * stride;
  float* xs = reinterpret_cast<float*>(codes + (blockDim.x >> 6) * stride) +
              wave * (a.chunk / kGroup);  // Block_FP8's
  constexpr int kLaneHeld = 2;  // pieces of eight hidden values a lane
  auto load_held = [&](Hidden (&h)[kLaneHeld], int c0) {
    const int cols = min(a.chunk, hi - c0), per = (cols + kGroup - 1) / kGroup * (kGroup / 8);
#pragma unroll
    for (int q = 0; q < kLaneHeld; ++q) {
      h[q] = Hidden{};
      if (lane + 64 * q < per) h[q] = load_hidden(a, &from, lane + 64 * q, per, c0, cols);
    }
  };
  int kb = lo / KSTEP;  // the chunk's first step
  auto last_step = [&](int c0) {
    return min((min(c0 + a.chunk, hi) + KSTEP - 1) / KSTEP, kfull);
  };
  Hidden held[kLaneHeld];
  load_held(held, lo);
  auto p = products<FMT, 1, 1, steps<FMT>(2), false>(
      kb, last_step(lo), [&](int, int k) -> Frag { return weight_step<FMT, PACKED>(wp, k); },
      [&](int, int k) -> Frag { return load_frag<FMT>(x + 16 * g, k - kb); },
      [&](int, int k) { return uniform_load(swp + k); }, [&](int, int k) { return xs[k - kb]; });
  p.begin();
  float sx = 0.0f, sw[4];
  if constexpr (!BLOCK) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sw[i] = swp[i];  // (used at the end)
    unsigned top = 0;
#pragma unroll
    for (int q = 0; q < kLaneHeld; ++q) top = max(top, largest(held[q]));
    for (int k = lo + 8 * (lane + 64 * kLaneHeld); k < hi; k += 512) {
      Hidden v;
      __builtin_memcpy(v.f, a.h + (long long)from * a.I + k, 32);
      top = max(top, largest(v));
    }
    top = wave_umax(top);
    if (a.parts > 1) {
      if (lane == 0) tops[wave] = top;
      __syncthreads();
      for (int w = 0; w < a.parts; ++w) top = max(top, tops[entry * a.parts + w]);
    }
    sx = act_scale<INT8>(__uint_as_float(top));
  }
  Acc acc[1][1] = {{Acc{0, 0, 0, 0}}};
  for (int c0 = lo; c0 < hi; c0 += a.chunk) {
    const int cols = min(a.chunk, hi - c0), per = (cols + kGroup - 1) / kGroup * (kGroup / 8);
    if (c0 > lo) {
      load_held(held, c0);
      p.la = kb = c0 / KSTEP;
      p.lfull = last_step(c0);
      p.begin();
    }
    auto encode = [&](Hidden v, int i) {
      const int k = 8 * i;
      float s = sx;
      if constexpr (BLOCK) {  // 16 lanes hold a group
        s = act_scale<false>(__uint_as_float(seg16_umax(largest(v))));
        if (k % kGroup == 0) xs[k / kGroup] = s;
      }
      *reinterpret_cast<v2u*>(x + k) = encode_values<INT8>(v.f, s, act_recip(s));
    };
    // (the wave's own LDS, which it accesses in order: the fences keep the
    // compiler from moving reads of the codes above the writes, and the next
    // chunk's writes above the reads)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
#pragma unroll
    for (int q = 0; q < kLaneHeld; ++q)
      if (lane + 64 * q < per) encode(held[q], lane + 64 * q);
    for (int i = lane + 64 * kLaneHeld; i < per; i += 64)
      encode(load_hidden(a, &from, i, per, c0, cols), i);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    p.run(acc);
    if constexpr (!BLOCK) {
      if (c0 + cols > kfull * KSTEP)
        p.multiply(acc[0][0], weight_tail<FMT, PACKED>(wp, kfull, a.I),
                   load_frag<FMT>(x + 16 * g, kfull - kb), 0.0f);
    }
  }
  // (every column of the product is the entry's)
  if ((lane & 15) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (!BLOCK) scales[entry][4 * g + i] = sx * sw[i];
      sums[wave][4 * g + i] = acc[0][0][i];
    }
  }
  if (lane == 0) {
    weights[entry] = weight;
    counts[entry] = on;
  }
  __syncthreads();
  if ((int)threadIdx.x < 16 * entries) {
    const int i = threadIdx.x / 16, c = threadIdx.x % 16;
    auto v = sums[i * a.parts][c];
    for (int w = 1; w < a.parts; ++w) v += sums[i * a.parts + w][c];
    float o = (float)v;
    if constexpr (!BLOCK) o *= scales[i][c];
    outputs[i][c] = o;
  }
  __syncthreads();
  if ((int)threadIdx.x < 16 * a.T) {
    const int t = threadIdx.x / 16, c = threadIdx.x % 16;
    float sum = a.base ? bf16_lo(a.base[t * a.ldb + n + c]) : 0.0f;
#pragma unroll 4
    for (int j = t * a.topk; j < (t + 1) * a.topk; ++j)
      sum = counts[j] ? __builtin_fmaf(weights[j], outputs[j][c], sum) : sum;
    a.y[t * a.ldy + n + c] = (uint16_t)bf16_bits(sum);
  }
}

template <int FMT, bool PACKED, int MB>
hipError_t launch_up(const MoeLayerArgs& a, hipStream_t s) {
  // Short K leaves four waves a step or two each: where there are columns enough
  // for every compute unit, a wave takes all of it (64 experts, top 8, I = 1024, 8
  // tokens in Block_FP8: D = 512 27.5 us and 22.9, 768 31.5 and 30.8, 1024 34.7 and
  // 37.6; in int8 28.0 and 23.5, 34.3 and 35.1, 38.2 and 42.3; 1 token, D = 768: 13.5
  // and 13.6).
  const int blocks = (a.I / 16 + kWaves - 1) / kWaves;
  if (a.D <= 768 && (long long)blocks * a.slots >= kComputeUnits)
    return launch_kernel(moe_up_kernel<FMT, PACKED, MB, 1>,
                         dim3((unsigned)blocks, (unsigned)a.slots), dim3(kThreads), 0, s, a);
  return launch_kernel(moe_up_kernel<FMT, PACKED, MB, kWaves>,
                       dim3((unsigned)(a.I / 16), (unsigned)a.slots), dim3(kThreads), 0, s, a);
}
template <int FMT, bool PACKED, int MB>
hipError_t launch_down(const MoeLayerArgs& a, hipStream_t s) {
  const size_t row = a.chunk + kPad + (FMT == BLOCK_FP8 ? a.chunk / kGroup * 4 : 0);
  if (MB == 1 && a.parts) {
    const int waves = a.T * a.topk * a.parts;
    return launch_kernel(moe_down_few_kernel<FMT, PACKED>, dim3((unsigned)(a.D / 16)),
                         dim3((unsigned)(64 * waves)), waves * row, s, a);
  }
  const dim3 grid((unsigned)((a.D + kColumns - 1) / kColumns), (unsigned)a.slots,
                  (unsigned)a.splits);
  if (!a.hq)
    return launch_kernel(moe_down_kernel<FMT, PACKED, MB, false>, grid, dim3(kThreads), a.T * row,
                         s, a);
  const int pieces = (a.I + 7) / 8, threads = min((pieces + 63) / 64 * 64, kEncodeThreads);
  const hipError_t e = launch_kernel(moe_encode_kernel<FMT>, dim3((unsigned)(a.T * a.topk)),
                                     dim3((unsigned)threads), 0, s, a);
  if (e != hipSuccess) return e;
  return launch_kernel(moe_down_kernel<FMT, PACKED, MB, true>, grid, dim3(kThreads), 0, s, a);
}
template <int FMT, int MB>
hipError_t launch_layer(bool packed1, bool packed2, const MoeLayerArgs& a, hipStream_t s) {
  const hipError_t e = packed1 ? launch_up<FMT, true, MB>(a, s) : launch_up<FMT, false, MB>(a, s);
  if (e != hipSuccess) return e;
  return packed2 ? launch_down<FMT, true, MB>(a, s) : launch_down<FMT, false, MB>(a, s);
}
// Experts of more than 16 tokens multiply two blocks of them by one weight (32
// tokens, 8 of 8 experts of 2048 x 4096: 72 us, a block at a time in the first kernel
// alone 80); calls without such experts are as fast either way (32 tokens, 2 of 8 of
// 4096 x 4096: 90.9), and calls that cannot have any need no registers for them.
template <int FMT>
hipError_t launch_layer(bool packed1, bool packed2, const MoeLayerArgs& a, hipStream_t s) {
  static_assert(kLayerTokens <= 32, "both kernels take all of an expert's tokens in two blocks");
  return a.T > 16 ? launch_layer<FMT, 2>(packed1, packed2, a, s)
                  : launch_layer<FMT, 1>(packed1, packed2, a, s);
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
