// Tiled Block_FP8 GEMM for any token count, dense and per expert.
//
//   Y[m, n] = sum_g sx[m, g] sw[n / 128, g] sum_{k in group g} Xq[m, k] Wq[n, k]
//
// A workgroup computes BM tokens x BN weight rows.  K advances by one 128-wide
// scale group per step.  Each step's codes (and the tokens' scales) go from
// memory straight into LDS by direct-to-LDS loads, ST steps deep, so they
// need no registers and stay in flight across the barrier; the waves read
// MFMA operands from LDS.  MFMA operand A is the weights and B the tokens
// (D = W X^T), so a lane's accumulators all belong to one token: the step's
// scale is one product per token column, and a group's partial sum is added
// as acc += partial * (sx * sw), one fp32 FMA per element per group.  The
// instruction itself rounds a group's sum: by 2^-16 of the result in the root
// mean square, unbiased, at most 2^-16 of the sum of |products| (measured, 2^17
// results), so about 1% of the bf16 outputs lie one step beside the rounded
// exact one; the fp32 sum over the groups adds nothing to that.
//
// Measured, and what bounds it: 8192 x 5120 x 8192 284 to 300 us, 2.3 to 2.4
// PFLOP/s, by power (0.555 M clocks at 1.7 .. 2.0 GHz) and the direct-to-LDS
// loads beside the MFMAs; 4096 x 5120 x 2048 46 us, 1.87 PFLOP/s, by the start
// and the output of a tile, which nothing on the compute unit overlaps; 48 x
// 4608 x 7168 12 us by the weights (5 us at the rate of reads, 7 at a copy's),
// the hand-off of split K and the start; 128 experts, top 8, of 1536 x 2048: 8
// tokens 33.5 us, 4.9 TB/s, by the weights' bytes; 4096 tokens 158 to 182 us
// (0.333 M clocks at 1.85 .. 2.1 GHz), 1.3 PFLOP/s, as the dense tiles.
#include <atomic>
#include <climits>
#include <type_traits>
#include <utility>

#include "w8_block.hpp"
#include "w8_device.hpp"
#include "w8_launch.hpp"
#include "w8_lds.hpp"

namespace w8 {
namespace {

// blockIdx -> work id such that each XCD (workgroups are dealt to the 8 XCDs
// in turn) runs one contiguous range of ids and its L2 sees neighbours.
__device__ __forceinline__ int xcd_contiguous(int b, int total) {
  const int q = total >> 3, r = total & 7, x = b & 7;
  return x * q + min(x, r) + (b >> 3);
}

template <int BM_, int BN_, int WM_, int WN_, int ST_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, ST = ST_;
  static constexpr int NW = WM * WN, THREADS = 64 * NW;
  static constexpr bool LARGE = false;
  // waves of a SIMD: two workgroups on a compute unit where LDS holds them
  static constexpr int WAVES = ST * (BM + BN) * 128 < 80 * 1024 ? NW / 2 : 2;
  static constexpr int NM = BM / WM / 16, NN = BN / WN / 16;  // MFMA tiles per wave
  static_assert(BN / WN <= 128, "a wave's weight rows lie in one 128-row scale block");
  // LDS: ST stages of token and weight codes, then two buffers of scales for
  // eight steps each: the tokens' (32 bytes a token), then the weight blocks'
  static constexpr int X_BYTES = BM * 128, W_BYTES = BN * 128;
  static constexpr int STAGE = X_BYTES + W_BYTES;
  static constexpr int SX_BYTES = (BM * 32 + 1023) / 1024 * 1024;
  static constexpr int SCALES = SX_BYTES + 256;
  static constexpr int LDS = ST * STAGE + 2 * SCALES;
  // direct-to-LDS loads of one wave per stage (a wave whose share is short
  // repeats its last piece, so that every wave counts the same loads)
  static constexpr int PX = (X_BYTES / 1024 + NW - 1) / NW;
  static constexpr int PW = (W_BYTES / 1024 + NW - 1) / NW;
  static constexpr int LOADS = PX + PW;
  // The large tiles run the rotated loop (see there): H weight tiles per half
  // step; the first H + 2 of a step are staged with its tokens, the others
  // one step later.  In LDS a stage's weight tiles (16 rows, 2 KiB) are
  // ordered early ones first.
  static constexpr bool ROTATED = NN * NM >= 16;
  static constexpr int H = NN / 2, EARLY = ROTATED ? H + 2 : NN;
  static_assert(!ROTATED || EARLY == NN || ST == 2, "late weight tiles follow one step behind");
  static constexpr int PW1 = WN * EARLY * 2 / NW;  // (exact where ROTATED)
  static __device__ __forceinline__ constexpr int slot(int wn, int i) {
    return i < EARLY ? wn * EARLY + i : WN * EARLY + wn * (NN - EARLY) + i - EARLY;
  }
  // the weight tile, counted from the workgroup's first, in slot u
  static __device__ __forceinline__ int tile_in(int u) {
    if (EARLY == NN) return u;
    if (u < WN * EARLY) return u / EARLY * NN + u % EARLY;
    constexpr int L = NN - EARLY > 0 ? NN - EARLY : 1;
    u -= WN * EARLY;
    return u / L * NN + EARLY + u % L;
  }
};

extern __shared__ __align__(1024) uint8_t smem[];

// As wait_stage() with the loads of n more steps (at most N) left in flight.
template <class T, int N>
__device__ __forceinline__ void wait_steps(int n) {
  if constexpr (N > 0) {
    if (n < N) return wait_steps<T, N - 1>(n);
  }
  wait_stage<N * T::LOADS>();
}

// f(0), f(1), ... as compile-time constants.
template <int... I, class F>
__device__ __forceinline__ void for_each_number(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}

// Vectors in memory at any address of a bf16 value: global stores need no more
// alignment than that, so rows of any length and leading dimension are written
// the same way.
typedef v4u v4u_any __attribute__((aligned(2)));
typedef v2u v2u_any __attribute__((aligned(2)));

// Four fp32 values to bf16, round to nearest even (NaN stays NaN).
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v2u bf16x4(v4f v) {
  return __builtin_bit_cast(v2u, __builtin_convertvector(v, bf16x4_t));
}

// One tile: rows [m0, m1) of Y (at most BM) times weight rows n0 .. n0 + BN - 1
// of the expert (wq, sw), over the K-steps [ks0, ks1); split and tile: which
// part of K of which output tile this is (split_k > 1).
template <class T, bool GROUPED, bool PACKED>
__device__ __forceinline__ void run_tile(const BlockGemmArgs& a, int m0, int m1, int n0,
                                         const uint8_t* wq, const float* sw, int ks0, int ks1,
                                         int split, int tile) {
  constexpr int BM = T::BM, BN = T::BN, NW = T::NW, NM = T::NM, NN = T::NN, ST = T::ST;
  // gathered token rows by pointer, except in the largest tile, which has no
  // registers for that (the host keeps rows more than 4 GiB apart from it)
  constexpr bool POINTERS = GROUPED && !T::LARGE;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % T::WM, wn = wave / T::WM;
  const int r = lane & 15, q = lane >> 4;

  // ---- this wave's load addresses.  Row-major pieces are 8 rows x 128 bytes,
  // lane i holding row i / 8; the 16-byte chunk it loads is rotated by an
  // exclusive-or with the row, so that the 16 rows of an operand read fall
  // into different LDS banks.  Rows past the end repeat the last one (their
  // products are not stored).
  const int prow = lane >> 3, pchunk = (lane & 7) ^ prow;
  const int k_steps = a.G;
  // a last step that K ends inside of: chunks past K re-read the last whole
  // one, and the tokens' are cleared in LDS (clear_tail)
  const int tail_chunks = (a.K & 127) >> 4;
  const int tail_step = tail_chunks ? k_steps - 1 : -2;  // (-2: none, nor is -1 before step 0)
  const int tail_adj = 16 * (min(pchunk, max(tail_chunks, 1) - 1) - pchunk);

  auto x_row = [&](int i) -> long long {
    const int m = min(m0 + i, m1 - 1);
    if constexpr (GROUPED) {
      if (a.rows) return min(max(a.rows[m], 0), a.xrow_max);
    }
    return m;
  };
  // Tokens: an offset from the tile's first row, for gathered rows from the
  // array's (which may lie more than 4 GiB apart: pointers).  Weights: an
  // offset from the tile's first row.  The bases advance by one step with each
  // step's loads.
  const uint8_t* px[T::PX];
  unsigned ox[T::PX], ow[T::PW];
  const uint8_t* xb = a.xq + 128LL * ks0;
  const uint8_t* wb = wq;
  if constexpr (!GROUPED) xb += m0 * a.ldq;
  if constexpr (PACKED)
    wb += ((long long)(n0 / 16) * k_steps + ks0) * 2048;
  else
    wb += n0 * a.ldw + 128LL * ks0;
#pragma unroll
  for (int i = 0; i < T::PX; ++i) {
    const int p = min(wave + i * NW, T::X_BYTES / 1024 - 1);
    if constexpr (POINTERS)
      px[i] = xb + x_row(8 * p + prow) * a.ldq + 16 * pchunk;
    else if constexpr (GROUPED)
      ox[i] = (unsigned)(x_row(8 * p + prow) * a.ldq + 16 * pchunk);
    else
      ox[i] = (unsigned)(min(8 * p + prow, m1 - 1 - m0) * a.ldq + 16 * pchunk);
  }
#pragma unroll
  for (int i = 0; i < T::PW; ++i) {
    const int p = min(wave + i * NW, T::W_BYTES / 1024 - 1);
    const int wt = T::tile_in(p / 2);
    if constexpr (PACKED)  // fragments of 16 rows x 128 bytes, 2 KiB per K-step, in lane order
      ow[i] = (unsigned)(min(wt, (a.N + 15) / 16 - 1 - n0 / 16) * k_steps) * 2048u +
              (p & 1) * 1024 + 16 * lane;
    else
      ow[i] = (unsigned)(min(16 * wt + 8 * (p & 1) + prow, a.N - 1 - n0) * a.ldw + 16 * pchunk);
  }
  const unsigned lds0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;

  // Token scales: 16 bytes (four steps) per lane, token 32 w + lane / 2 by
  // wave w.  Near the end of a row the four are its last four (scales()
  // knows); a row of fewer than four goes in single words.
  const int G = a.G;
  const float* swt = sw + (long long)(n0 / 128) * G;
  const int sw_blocks = min((a.N + 127) / 128 - n0 / 128, (BN + 127) / 128);
  static_assert(T::SX_BYTES / 1024 <= NW, "a wave loads one piece of the token scales");
  const float* sxt = a.sx + x_row(min(32 * wave + (lane >> 1), BM - 1)) * G;
  auto scale_start = [&](int g4) { return G >= 4 ? min(g4, G - 4) : g4; };
  auto issue_scales = [&](int c) {
    const unsigned base = lds0 + ST * T::STAGE + (c & 1) * T::SCALES;
    if (G >= 4) {
      if (wave < T::SX_BYTES / 1024)
        load_lds16(reinterpret_cast<const uint8_t*>(sxt + scale_start(8 * c + 4 * (lane & 1))),
                   base + wave * 1024);
    } else {
      for (int p = wave; p < T::SX_BYTES / 256; p += NW)
        load_lds4(a.sx + x_row(min(8 * p + (lane >> 3), BM - 1)) * G + min(lane & 7, G - 1),
                  base + p * 256);
    }
    if (wave == NW - 1)
      load_lds4(swt + (long long)min((lane >> 3) & 1, sw_blocks - 1) * G +
                    min(8 * c + (lane & 7), G - 1),
                base + T::SX_BYTES);
  };

  // load n (compile time) of the wave's share of a step, into the stage at LDS
  // address `base`; the late weight tiles (ROTATED) are the previous step's,
  // into the stage at `late`
  const uint8_t* wb_late = wb;
  auto issue_one = [&](int n, unsigned base, unsigned late) {
    if (n < T::PX) {
      const unsigned lds = base + min(wave + n * NW, T::X_BYTES / 1024 - 1) * 1024;
      if constexpr (POINTERS)
        load_lds16(px[n], lds);
      else
        load_lds16(xb, ox[n], lds);
    } else {
      const int i = n - T::PX;
      const bool is_late = T::ROTATED && i >= T::PW1;
      load_lds16(is_late ? wb_late : wb, ow[i],
                 (is_late ? late : base) + T::X_BYTES +
                     min(wave + i * NW, T::W_BYTES / 1024 - 1) * 1024);
    }
  };
  auto advance_bases = [&] {
    if constexpr (POINTERS) {
#pragma unroll
      for (int i = 0; i < T::PX; ++i) px[i] += 128;
    } else {
      xb += 128;
    }
    wb += PACKED ? 2048 : 128;
  };
  // Before the loads of step k (in order): moves the bases on from step k - 1,
  // and at the step that K ends inside of moves the lanes off the missing
  // chunks.  (ROTATED: past the last step the bases stay, and its loads go into
  // a stage that nobody reads.)
  // Scales of steps 8c .. 8c + 7 come with the first step that needs them: a
  // token's scales are consecutive in memory, so taking eight steps at once
  // fetches each cache line an eighth as often as one step would.
  auto advance = [&](int k) {
    if constexpr (T::ROTATED && T::PW1 < T::PW) {
      if (k > ks0 + 1) wb_late += PACKED ? 2048 : 128;
      if (k - 1 == tail_step) {
#pragma unroll
        for (int i = T::PW1; i < T::PW; ++i) ow[i] += tail_adj;
      }
    }
    if (k >= ks1) return;
    if (k > ks0) advance_bases();
    if (k == tail_step) {
#pragma unroll
      for (int i = 0; i < T::PX; ++i) {
        if constexpr (POINTERS)
          px[i] += tail_adj;
        else
          ox[i] += tail_adj;
      }
#pragma unroll
      for (int i = 0; i < (T::ROTATED ? T::PW1 : T::PW); ++i) ow[i] += tail_adj;
    }
    if ((k & 7) == 0 || k == ks0) issue_scales(k >> 3);
  };

  v4f acc[NN][NM];
#pragma unroll
  for (int i = 0; i < NN; ++i)
#pragma unroll
    for (int j = 0; j < NM; ++j) acc[i][j] = v4f{0, 0, 0, 0};

  // ---- LDS reads
  const int c0 = 16 * (q ^ (r & 7)), c1 = 16 * ((q + 4) ^ (r & 7));
  auto frag = [&](const uint8_t* p, int off0, int off1) -> v8i {
    const v4i lo = *reinterpret_cast<const v4i*>(p + off0);
    const v4i hi = *reinterpret_cast<const v4i*>(p + off1);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto tokens = [&](int j, int stage) {
    return frag(smem + stage * T::STAGE + (wm * NM + j) * 2048, r * 128 + c0, r * 128 + c1);
  };
  auto weights = [&](int i, int stage) {
    const uint8_t* p = smem + stage * T::STAGE + T::X_BYTES + T::slot(wn, i) * 2048;
    return PACKED ? frag(p, 16 * lane, 1024 + 16 * lane) : frag(p, r * 128 + c0, r * 128 + c1);
  };
  // the tokens' scales of step k times the weight block's (a row's last four
  // scales lie `last_shift` bytes on where G is no multiple of four)
  const int last_four = G >= 4 && G % 4 ? G & ~3 : INT_MAX, last_shift = 4 * (4 - G % 4);
  const uint8_t* ssx = smem + ST * T::STAGE + (wm * 16 * NM + r) * 32;
  const uint8_t* ssw = smem + ST * T::STAGE + T::SX_BYTES + 32 * ((wn * 16 * NN) / 128);
  auto scales = [&](int k, float* sc) {
    const int o = (k & 8 ? T::SCALES : 0) + 4 * (k & 7);
    const float swk = *reinterpret_cast<const float*>(ssw + o);
    const uint8_t* sx = ssx + (o + (k >= last_four ? last_shift : 0));
#pragma unroll
    for (int j = 0; j < NM; ++j) sc[j] = *reinterpret_cast<const float*>(sx + 512 * j) * swk;
  };
  // where K ends inside step k: the tokens' chunks past it become zeros
  auto clear_tail = [&](int stage) {
    uint8_t* xs = smem + stage * T::STAGE;
    for (int c = threadIdx.x; c < BM * (8 - tail_chunks); c += T::THREADS) {
      const int row = c / (8 - tail_chunks), ch = tail_chunks + c % (8 - tail_chunks);
      *reinterpret_cast<v4i*>(xs + row * 128 + 16 * (ch ^ (row & 7))) = v4i{0, 0, 0, 0};
    }
    wait_stage<63>();
  };

  // MFMA n goes out while the scaled additions of MFMA n - LAG, whose result
  // has arrived, run beside it; the scheduling barriers keep the compiler from
  // pairing each MFMA with its own additions, which would wait out its latency
  // every time.  A step's loads are dealt over its first MFMAs: all at once
  // they would hold up the MFMAs behind the memory path's queue, and later
  // they would arrive after the step's end (8192 x 5120 x 8192 on the largest
  // tile: one load every two MFMAs 300 us, one a MFMA 307, one every three
  // 304 to 311).
  constexpr int LAG = NN * NM < 4 ? 1 : 3;
  constexpr int P = NN * NM;
  v4f t[LAG + 1];
  typedef std::integral_constant<bool, true> Yes;
  typedef std::integral_constant<bool, false> No;
  if constexpr (T::ROTATED) {
    // The loop is rotated by half a step against the staging: between two
    // barriers the waves run the second half of step k - 1 (weight tiles H ..
    // NN - 1) and the first half of step k.  At a barrier the registers hold
    // the operands of the next MFMAs, and the tokens of step k replace those
    // of step k - 1 one by one inside the interval, so that no wave waits for
    // operand reads behind a barrier, and every load has a whole interval to
    // arrive.  The last two weight tiles of a step run side by side, which
    // frees the first token operand early.
    constexpr int H = T::H, P2 = (NN - H) * NM, PJ = P2 - 2 * NM;
    v8i wf[4], xf[NM];
    float sc0[NM], sc1[NM];  // of steps k - 1 and k
    auto tile_of = [](int p) constexpr {
      return p >= P2 ? (p - P2) / NM : p < PJ ? H + p / NM : NN - 2 + (p & 1);
    };
    auto j_of = [](int p) constexpr {
      return p >= P2 || p < PJ ? p % NM : (p - PJ) / 2;
    };
    auto add = [&](int p, const float* sc) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        acc[tile_of(p)][j_of(p)][u] =
            __builtin_fmaf(t[p % 4][u], sc[j_of(p)], acc[tile_of(p)][j_of(p)][u]);
    };
    static_assert(P % 4 == 0 && NM % 4 == 0, "the ring of partial results continues over intervals");
    auto interval = [&](auto first, auto last, int k, int stage) {
      constexpr bool FIRST = decltype(first)::value, LAST = decltype(last)::value;
      wait_stage<(ST - 2) * T::LOADS>();
      if (!LAST && k == tail_step) clear_tail(stage);
      if constexpr (!LAST) advance(k + ST - 1);
      const int before = stage == 0 ? ST - 1 : stage - 1;  // the stage of step k - 1
      const unsigned here = lds0 + stage * T::STAGE, other = lds0 + before * T::STAGE;
      if constexpr (FIRST) {
        wf[0] = weights(0, stage);
#pragma unroll
        for (int j = 0; j < NM; ++j) xf[j] = tokens(j, stage);
        wf[1] = weights(1, stage);
        scales(k, sc1);
      }
#pragma unroll
      for (int p = FIRST ? P2 : 0; p < (LAST ? P2 : P); ++p) {
        if constexpr (!FIRST) {
          if (p < (NN - H - 2) * NM && p % NM == 0)  // (their slots' tiles are done)
            wf[(H + 2 + p / NM) % 4] = weights(H + 2 + p / NM, before);
          if constexpr (!LAST) {
            if (p == PJ) {
              scales(k, sc1);
              wf[0] = weights(0, stage);
            }
            if (p == PJ + 2) wf[1] = weights(1, stage);
          }
        }
        if (p >= P2 && (p - P2) % NM == 0) {
          const int i = (p - P2) / NM + 2;
          if (i < T::EARLY) wf[i % 4] = weights(i, stage);
        }
        if constexpr (!LAST) {
          // (every other MFMA where a whole step is left to deal them)
          const int n = p - (FIRST ? P2 : 0), gap = FIRST ? 1 : 2;
          if (n % gap == 0 && n / gap < T::LOADS) issue_one(n / gap, other, here);
        }
        t[p % 4] = mfma_f8(wf[tile_of(p) % 4], xf[j_of(p)], v4f{0, 0, 0, 0});
        if (!FIRST && !LAST && p >= PJ && p < P2 && (p & 1)) xf[j_of(p)] = tokens(j_of(p), stage);
        if (p >= LAG + (FIRST ? P2 : 0))
          add(p - LAG, p - LAG >= P2 ? sc1 : sc0);
        else if (!FIRST)
          add(P + p - LAG, sc0);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (LAST) {
#pragma unroll
        for (int p = P2 - LAG; p < P2; ++p) add(p, sc0);
      } else {
#pragma unroll
        for (int j = 0; j < NM; ++j) sc0[j] = sc1[j];
      }
    };
    static_assert(P - P2 >= T::LOADS && P >= 2 * T::LOADS, "an interval deals all loads");
    // (no late weight tiles here: there is no step before the first, and where
    // K ends inside that one their offsets still point past the rows' ends)
#pragma unroll
    for (int s = 0; s < ST - 1; ++s) {
      advance(ks0 + s);
#pragma unroll
      for (int n = 0; n < T::PX + T::PW1; ++n)
        issue_one(n, lds0 + s * T::STAGE, lds0 + (s + 1) * T::STAGE);
    }
    interval(Yes{}, No{}, ks0, 0);
    int stage = 1;
    for (int k = ks0 + 1; k < ks1; ++k) {
      interval(No{}, No{}, k, stage);
      stage = stage == ST - 1 ? 0 : stage + 1;
    }
    interval(No{}, Yes{}, ks1, stage);
  } else {
    // Operands are read one step ahead, into a second register set, between
    // the MFMAs: past the barrier of step k every wave holds that step's
    // operands, its stage is loaded with step k + ST, and step k + 1 is read.
    // What bounds these tiles is the instructions of a wave, one in four
    // clocks, beside the MFMAs; so the steps run in groups whose stages and
    // register sets are constants (128 x 128: 935 clocks a step, 512 of them
    // MFMAs; with the operands read behind the barrier and the stage a
    // variable 1240).
    constexpr int GROUP = ST % 2 ? 2 * ST : ST, F = NM + NN;
    static_assert(ST + GROUP + 1 <= 10, "no scales land on those still to be read");
    static_assert(P % (LAG + 1) == 0, "the ring of partial results continues over steps");
    v8i wf[2][NN], xf[2][NM];
    float sc[2][NM];
    auto read = [&](int f, int stage, int set) {  // fragment f, in the order of use
      if (f == 0)
        wf[set][0] = weights(0, stage);
      else if (f <= NM)
        xf[set][f - 1] = tokens(f - 1, stage);
      else
        wf[set][f - NM] = weights(f - NM, stage);
    };
    auto add = [&](int n, int set) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        acc[n / NM][n % NM][u] =
            __builtin_fmaf(t[n % (LAG + 1)][u], sc[set][n % NM], acc[n / NM][n % NM][u]);
    };
    auto issue_step = [&](int stage) {
#pragma unroll
      for (int n = 0; n < T::LOADS; ++n) issue_one(n, lds0 + stage * T::STAGE, 0);
    };
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      if (ks0 + s >= ks1) break;
      advance(ks0 + s);
      issue_step(s);
    }
    wait_steps<T, ST - 1>(ks1 - 1 - ks0);
    if (ks0 == tail_step) clear_tail(0);
#pragma unroll
    for (int f = 0; f < F; ++f) read(f, 0, 0);
    scales(ks0, sc[0]);
#pragma unroll
    for (int j = 0; j < NM; ++j) sc[1][j] = 0.0f;
#pragma unroll
    for (int n = 0; n < LAG + 1; ++n) t[n] = v4f{0, 0, 0, 0};
    int k = ks0;
    // Groups that load whole steps only.  The additions of a step's last MFMAs
    // run beside the next step's first (before the first step: of zeros).
    for (const int end = min(ks1, tail_step >= 0 ? tail_step : ks1) - (ST + GROUP); k <= end;
         k += GROUP) {
#pragma unroll
      for (int s = 0; s < GROUP; ++s) {
        const int stage = s % ST, set = s % 2;
        wait_stage<(ST - 2) * T::LOADS>();  // steps k + s + 2 .. k + s + ST - 1 are in flight
        // the scales that the group's loads come to need
        if (s == 0 && ((k + ST - 1) & 8) != ((k + ST + GROUP - 1) & 8))
          issue_scales((k + ST + GROUP - 1) >> 3);
        advance_bases();
#pragma unroll
        for (int n = 0; n < P; ++n) {
#pragma unroll
          for (int l = n * T::LOADS / P; l < (n + 1) * T::LOADS / P; ++l)
            issue_one(l, lds0 + stage * T::STAGE, 0);
#pragma unroll
          for (int f = n * F / P; f < (n + 1) * F / P; ++f) read(f, (s + 1) % ST, set ^ 1);
          t[n % (LAG + 1)] = mfma_f8(wf[set][n / NM], xf[set][n % NM], v4f{0, 0, 0, 0});
          if (n >= LAG)
            add(n - LAG, set);
          else
            add(P + n - LAG, set ^ 1);
          if (n == LAG) scales(k + s + 1, sc[set ^ 1]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
#pragma unroll
    for (int n = P - LAG; n < P; ++n) add(n, 1);
    // the steps that are left, at most ST + GROUP
    auto step = [&](auto number) {
      if (k >= ks1) return;
      constexpr int s = decltype(number)::value, stage = s % ST, next = (s + 1) % ST, set = s % 2;
      if (k + 1 < ks1) wait_steps<T, ST - 2>(min(ks1 - 2 - k, ST - 2));
      if (k + ST < ks1) {
        advance(k + ST);
        issue_step(stage);
      }
      if (k + 1 == tail_step) clear_tail(next);
      // (past the last step these read what nobody uses)
#pragma unroll
      for (int n = 0; n < P; ++n) {
#pragma unroll
        for (int f = n * F / P; f < (n + 1) * F / P; ++f) read(f, next, set ^ 1);
        t[n % (LAG + 1)] = mfma_f8(wf[set][n / NM], xf[set][n % NM], v4f{0, 0, 0, 0});
        if (n >= LAG) add(n - LAG, set);
        __builtin_amdgcn_sched_barrier(0);
      }
      scales(k + 1, sc[set ^ 1]);
#pragma unroll
      for (int n = P - LAG; n < P; ++n) add(n, set);
      ++k;
    };
    for_each_number(std::make_integer_sequence<int, ST + GROUP>{}, step);
  }
  wait_stage<0>();  // the loads past the last step have landed before LDS is used again or freed

  // ---- split-K: see the protocol of the small-M GEMM's shared tiles
  // (partials written through with agent scope, acknowledged, counted; the
  // last workgroup of the tile sums them in K order).
  if (!GROUPED && !T::LARGE && a.split_k > 1) {
    const int bytes = a.split_k * NW * NN * NM * 1024;
    const __amdgpu_buffer_rsrc_t prs =
        coherent_rsrc(reinterpret_cast<char*>(a.part) + (long long)tile * bytes, bytes);
    auto foff = [&](int s, int i, int j) {
      return (((s * NW + wave) * NN + i) * NM + j) * 1024 + 16 * lane;
    };
#pragma unroll
    for (int i = 0; i < NN; ++i)
#pragma unroll
      for (int j = 0; j < NM; ++j)
        coherent_store16(prs, foff(split, i, j), __builtin_bit_cast(v4i, acc[i][j]));
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __syncthreads();
    // (past the output tile, which the first waves write below while others
    // may not have read the flag yet)
    int* flag = reinterpret_cast<int*>(smem + T::LDS - 16);
    if (threadIdx.x == 0) {
      const unsigned inc = 256u / (unsigned)a.split_k;
      const unsigned prev = __hip_atomic_fetch_add(a.counters + (long long)tile * kCounterWords,
                                                   inc, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      *flag = ((prev + inc) & 255u) == 0u;
    }
    __syncthreads();
    if (!*flag) return;
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    // slots in batches whose loads are all in flight together, added in slot
    // order (a batch of the tile's 4 NN NM registers a slot, 64 at most)
    constexpr int Q = NN * NM >= 16 ? 1 : 16 / (NN * NM);
#pragma unroll
    for (int i = 0; i < NN; ++i)
#pragma unroll
      for (int j = 0; j < NM; ++j) acc[i][j] = v4f{0, 0, 0, 0};
    for (int s0 = 0; s0 < a.split_k; s0 += Q) {
      v4i v[Q][NN][NM];
#pragma unroll
      for (int s = 0; s < Q; ++s)
        if (s0 + s < a.split_k) {
#pragma unroll
          for (int i = 0; i < NN; ++i)
#pragma unroll
            for (int j = 0; j < NM; ++j) v[s][i][j] = coherent_load16(prs, foff(s0 + s, i, j));
        }
#pragma unroll
      for (int s = 0; s < Q; ++s)
        if (s0 + s < a.split_k) {
#pragma unroll
          for (int i = 0; i < NN; ++i)
#pragma unroll
            for (int j = 0; j < NM; ++j) acc[i][j] += __builtin_bit_cast(v4f, v[s][i][j]);
        }
    }
  }

  // ---- epilogue: lane (r, q) of tile (i, j) holds token 16 j + r, weight
  // rows 16 i + 4 q .. + 3
  if constexpr (BM * BN >= 128 * 128) {
    // through LDS, so that a store covers whole rows of the tile: 8-byte
    // stores of each lane's own four would touch 16 rows at a time (all
    // outputs of a 256 x 256 round take 8500 clocks, the rate of the writes)
    constexpr int ROW = BN * 2 + 32;
    static_assert(BM * ROW <= T::LDS - 16, "the output tile fits where the stages were");
#pragma unroll
    for (int j = 0; j < NM; ++j)
#pragma unroll
      for (int i = 0; i < NN; ++i)
        *reinterpret_cast<v2u*>(smem + ((wm * NM + j) * 16 + r) * ROW +
                                ((wn * NN + i) * 16 + 4 * q) * 2) = bf16x4(acc[i][j]);
    __syncthreads();
    // (a thread's column is the same every time: THREADS is a multiple of the
    // chunks of a row; the reads of a batch are in flight together)
    constexpr int CHUNKS = BN / 8, STEP = T::THREADS / CHUNKS;
    constexpr int BATCH = BM / STEP < 8 ? BM / STEP : 8;
    static_assert(T::THREADS % CHUNKS == 0 && BM % (STEP * BATCH) == 0, "whole batches");
    const int col = threadIdx.x % CHUNKS * 8, n = n0 + col;
    uint16_t* yp = a.y + (long long)m0 * a.ldy + n;
    const bool whole = n + 8 <= a.N;
    for (int r0 = threadIdx.x / CHUNKS; r0 < m1 - m0; r0 += STEP * BATCH) {
      v4u v[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b)
        v[b] = *reinterpret_cast<const v4u*>(smem + (r0 + b * STEP) * ROW + col * 2);
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int row = r0 + b * STEP;
        if (row >= m1 - m0) break;
        uint16_t* p = yp + row * a.ldy;
        if (whole) {
          // (the largest tile's outputs would push the operands out of L2:
          // non-temporal, 8192 x 5120 x 8192 301 -> 295 us)
          if constexpr (T::LARGE)
            __builtin_nontemporal_store(v[b], reinterpret_cast<v4u_any*>(p));
          else
            *reinterpret_cast<v4u_any*>(p) = v[b];
        } else {
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (n + u < a.N) p[u] = (uint16_t)(v[b][u >> 1] >> (16 * (u & 1)));
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NM; ++j) {
      const int m = m0 + (wm * NM + j) * 16 + r;
      if (m < m1) {
        uint16_t* yr = a.y + m * a.ldy;
#pragma unroll
        for (int i = 0; i < NN; ++i) {
          const int n = n0 + (wn * NN + i) * 16 + 4 * q;
          const v2u v = bf16x4(acc[i][j]);
          if (n + 4 <= a.N) {
            *reinterpret_cast<v2u_any*>(yr + n) = v;
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (n + u < a.N) yr[n + u] = (uint16_t)(v[u >> 1] >> (16 * (u & 1)));
          }
        }
      }
    }
  }
}

// The workgroup's part of K: steps [ks0, ks1).
struct KRange {
  int ks0, ks1;
};
__device__ __forceinline__ KRange k_range(const BlockGemmArgs& a, int split) {
  const int shift = __builtin_ctz(a.split_k);
  return {(int)((long long)a.G * split >> shift), (int)((long long)a.G * (split + 1) >> shift)};
}

// Which tile a workgroup of the dense GEMM takes: bands of 4 token tiles,
// weight tiles inside a band in order, so that the ids an XCD runs at one time
// form a near-square patch of tiles (4096 x 5120 x 2048: bands of 4 47.3 us, of
// 8 48.7, of 16 50.9).
struct TilePos {
  int tm, tn;
};
__device__ __forceinline__ TilePos tile_pos(const BlockGemmArgs& a, int id) {
  if (a.tiles_m == 1) return {0, id};
  const int band = 4 * a.tiles_n;
  const int b0 = id / band * 4;
  const int h = min(4, a.tiles_m - b0);
  return {b0 + id % band % h, id % band / h};
}

template <class T, bool PACKED>
__global__ __launch_bounds__(T::THREADS, T::WAVES) void block_gemm_kernel(BlockGemmArgs a) {
  if constexpr (T::LARGE) {
    // The tiles that fill whole rounds of the compute units run at full size;
    // those of the last, partial round (from id a.whole on) as two halves or
    // four quarters each (a.parts), so that the round gets shorter.  A tile
    // with at most 128 rows left runs at half height too.
    typedef typename T::Half Half;
    typedef typename T::Quarter Quarter;
    int id = blockIdx.x, part = 0;
    const bool whole = id < a.whole;
    if (whole) {
      id = xcd_contiguous(id, a.whole);
    } else {
      id = xcd_contiguous(id - a.whole, gridDim.x - a.whole);
      part = id & (a.parts - 1);
      id = a.whole + (id >> (a.parts >> 1));
    }
    const TilePos t = tile_pos(a, id);
    const int m0 = t.tm * T::BM + (part & 1) * Half::BM;
    const int m1 = min(m0 + (whole ? T::BM : Half::BM), a.M);
    const int n0 = t.tn * T::BN + (part >> 1) * Quarter::BN;
    if (m0 >= m1 || n0 >= a.N) return;
    if (whole && m1 - m0 > Half::BM)
      run_tile<T, false, PACKED>(a, m0, m1, n0, a.wq, a.sw, 0, a.G, 0, 0);
    else if (whole || a.parts == 2)
      run_tile<Half, false, PACKED>(a, m0, m1, n0, a.wq, a.sw, 0, a.G, 0, 0);
    else
      run_tile<Quarter, false, PACKED>(a, m0, m1, n0, a.wq, a.sw, 0, a.G, 0, 0);
  } else {
    const int work = xcd_contiguous(blockIdx.x, gridDim.x);
    const int split = work & (a.split_k - 1), tile = work >> __builtin_ctz(a.split_k);
    const TilePos t = tile_pos(a, tile);
    const KRange k = k_range(a, split);
    run_tile<T, false, PACKED>(a, t.tm * T::BM, min(t.tm * T::BM + T::BM, a.M), t.tn * T::BN, a.wq,
                               a.sw, k.ks0, k.ks1, split, tile);
  }
}

// Inclusive sum over the lanes of a wavefront: within rows of 16 lanes by
// shifts, then the rows' totals passed on (gfx9 DPP row_shr and row_bcast).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// Expert e has ceil(count / BM) token tiles; slot s is the s-th of them over
// all experts, found by every wave from the offsets.  The launch holds the
// most slots that n_rows entries can need, M / BM + min(E, M); those past the
// last tile exit at once.
template <class T, bool PACKED>
__global__ __launch_bounds__(T::THREADS, T::WAVES) void grouped_gemm_kernel(BlockGemmArgs a) {
  const int lane = threadIdx.x & 63;
  // Lane l holds experts e0 + 4 l .. + 3 of 256 at a time: the tiles of each,
  // and their running sum over the lanes.
  int off[5], tiles[4], sum = 0;
  auto scan = [&](int e0) {
#pragma unroll
    for (int i = 0; i < 5; ++i)
      off[i] = min(max(a.offsets[min(e0 + 4 * lane + i, a.n_experts)], 0), a.M);
    int mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tiles[i] = (max(off[i + 1] - off[i], 0) + T::BM - 1) / T::BM;
      mine += tiles[i];
    }
    sum = wave_scan(mine);
  };
  // the XCDs share the tiles there are, not the slots of the launch (which
  // bound them, whatever the offsets hold)
  int total = 0;
  for (int e0 = 0; e0 < a.n_experts; e0 += 256) {
    scan(e0);
    total = min(total + __builtin_amdgcn_readlane(sum, 63), a.tiles_m);
  }
  total *= a.tiles_n;
  int work = blockIdx.x, part = 0, parts = 1, whole = total;
  if constexpr (T::LARGE) {
    // a last, partial round in pieces, as in the dense kernel (the launch holds
    // kGroupedPieces workgroups more than slots for them)
    parts = last_round_parts(total);
    whole = parts > 1 ? total / kComputeUnits * kComputeUnits : total;
  }
  if (work < whole) {
    work = xcd_contiguous(work, whole);
    parts = 1;
  } else {
    work -= whole;
    const int pieces = (total - whole) * parts;
    if (work >= pieces) return;
    work = xcd_contiguous(work, pieces);
    part = work & (parts - 1);
    work = whole + (work >> (parts >> 1));
  }
  int n0 = work % a.tiles_n * T::BN;
  int slot = work / a.tiles_n, e = -1, lo = 0, hi = 0;
  for (int e0 = 0; e0 < a.n_experts; e0 += 256) {
    if (a.n_experts > 256) scan(e0);
    const unsigned long long past = __ballot(sum > slot);
    if (past) {
      const int l = __builtin_ctzll(past);
      slot -= l ? __builtin_amdgcn_readlane(sum, l - 1) : 0;
      // which of the lane's four
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = __builtin_amdgcn_readlane(tiles[i], l);
        if (e < 0 && slot < t) {
          e = e0 + 4 * l + i;
          lo = __builtin_amdgcn_readlane(off[i], l);
          hi = __builtin_amdgcn_readlane(off[i + 1], l);
        }
        if (e < 0) slot -= t;
      }
      break;
    }
    slot -= __builtin_amdgcn_readlane(sum, 63);
  }
  if (e < 0) return;
  int m0 = lo + slot * T::BM, m1 = min(m0 + T::BM, hi);
  const uint8_t* wq = a.wq + (long long)e * a.w_stride;
  const float* sw = a.sw + (long long)e * a.sw_stride;
  if constexpr (T::LARGE) {
    typedef typename T::Half Half;
    typedef typename T::Quarter Quarter;
    if (parts > 1) {
      m0 += (part & 1) * Half::BM;
      m1 = min(m0 + Half::BM, m1);
      n0 += (part >> 1) * Quarter::BN;
      if (m0 >= m1 || n0 >= a.N) return;
    }
    if (parts == 4) {
      run_tile<Quarter, true, PACKED>(a, m0, m1, n0, wq, sw, 0, a.G, 0, 0);
      return;
    }
    if (m1 - m0 <= Half::BM) {
      run_tile<Half, true, PACKED>(a, m0, m1, n0, wq, sw, 0, a.G, 0, 0);
      return;
    }
  }
  run_tile<T, true, PACKED>(a, m0, m1, n0, wq, sw, 0, a.G, 0, 0);
}

// The small tiles leave a compute unit room for two workgroups; stages that
// take all of LDS for one workgroup measured 2 to 3% slower.
typedef Tile<16, 128, 1, 4, 4> T0;
typedef Tile<64, 64, 2, 2, 4> T1;
typedef Tile<64, 128, 2, 4, 3> T2;
typedef Tile<128, 128, 4, 2, 4> T3;
struct T4 : Tile<256, 256, 4, 2, 2> {
  static constexpr bool LARGE = true;
  struct Half : Tile<128, 256, 2, 4, 3> {
    static constexpr bool LARGE = true;
  };
  struct Quarter : Tile<128, 128, 4, 2, 4> {
    static constexpr bool LARGE = true;
  };
  static constexpr int LDS = Half::LDS > Tile::LDS ? Half::LDS : Tile::LDS;
  static_assert(Quarter::LDS <= LDS, "");
};

template <class T>
constexpr BlockTile describe() {
  return BlockTile{T::BM, T::BN, T::THREADS, T::LDS};
}
const BlockTile kTiles[kBlockTiles] = {describe<T0>(), describe<T1>(), describe<T2>(),
                                       describe<T3>(), describe<T4>()};

typedef void (*Kernel)(BlockGemmArgs);

template <class T, Kernel K>
hipError_t launch(unsigned wgs, const BlockGemmArgs& a, hipStream_t s) {
  // more than 64 KiB of LDS has to be asked for, once per kernel and device
  // (the caller has checked that the device's number is below 64)
  static std::atomic<unsigned long long> asked{0};
  int device = 0;
  hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return e;
  if (!(asked.load(std::memory_order_relaxed) >> device & 1)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(K),
                            hipFuncAttributeMaxDynamicSharedMemorySize, T::LDS);
    if (e != hipSuccess) return e;
    asked.fetch_or(1ull << device, std::memory_order_relaxed);
  }
  return launch_kernel(K, dim3(wgs), dim3(T::THREADS), T::LDS, s, a);
}

template <class T>
hipError_t launch_dense(unsigned wgs, bool packed, const BlockGemmArgs& a, hipStream_t s) {
  return packed ? launch<T, block_gemm_kernel<T, true>>(wgs, a, s)
                : launch<T, block_gemm_kernel<T, false>>(wgs, a, s);
}
template <class T>
hipError_t launch_grouped(unsigned wgs, bool packed, const BlockGemmArgs& a, hipStream_t s) {
  return packed ? launch<T, grouped_gemm_kernel<T, true>>(wgs, a, s)
                : launch<T, grouped_gemm_kernel<T, false>>(wgs, a, s);
}
}  // namespace

const BlockTile& block_tile(int tile) { return kTiles[tile]; }

hipError_t launch_block_gemm(int tile, unsigned wgs, bool packed, const BlockGemmArgs& a,
                             hipStream_t s) {
  switch (tile) {
    case kTile16x128: return launch_dense<T0>(wgs, packed, a, s);
    case kTile64x64: return launch_dense<T1>(wgs, packed, a, s);
    case kTile64x128: return launch_dense<T2>(wgs, packed, a, s);
    case kTile128x128: return launch_dense<T3>(wgs, packed, a, s);
    case kTile256x256: return launch_dense<T4>(wgs, packed, a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_grouped_gemm(int tile, unsigned wgs, bool packed, const BlockGemmArgs& a,
                               hipStream_t s) {
  switch (tile) {
    case kTile16x128: return launch_grouped<T0>(wgs, packed, a, s);
    case kTile64x128: return launch_grouped<T2>(wgs, packed, a, s);
    case kTile128x128: return launch_grouped<T3>(wgs, packed, a, s);
    case kTile256x256: return launch_grouped<T4>(wgs, packed, a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace w8
