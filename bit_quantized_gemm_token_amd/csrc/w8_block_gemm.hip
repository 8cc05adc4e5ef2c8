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
// as acc += partial * (sx * sw), one fp32 FMA per element per group.
#include "w8_block.hpp"
#include "w8_device.hpp"
#include "w8_launch.hpp"

namespace w8 {
namespace {

// ------------------------------------------------------------ LDS traffic --
// Direct-to-LDS loads: lane i's 16 (or 4) bytes go to LDS byte lds + 16 i (or
// 4 i).  M0 carries the LDS address and needs one wait state before its use.
// Written as assembly because the compiler, which cannot tell the stages of
// the LDS buffer apart, would wait for every load in flight before each LDS
// read; wait_stage() below does the waiting.
__device__ __forceinline__ void load_lds16(const uint8_t* p, unsigned lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(lds), "v"(p)
               : "memory");
}
__device__ __forceinline__ void load_lds4(const float* p, unsigned lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(lds), "v"(p)
               : "memory");
}
// Waits until at most N of this wave's loads are in flight and its LDS reads
// have returned, then for the workgroup's other waves.
template <int N>
__device__ __forceinline__ void wait_stage() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

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
};

extern __shared__ __align__(1024) uint8_t smem[];

template <class T, bool GROUPED, bool PACKED>
__global__ __launch_bounds__(T::THREADS) void block_gemm_kernel(BlockGemmArgs a) {
  constexpr int BM = T::BM, BN = T::BN, NW = T::NW, NM = T::NM, NN = T::NN, ST = T::ST;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % T::WM, wn = wave / T::WM;
  const int r = lane & 15, q = lane >> 4;

  // ---- which tile
  int work = xcd_contiguous(blockIdx.x, gridDim.x);
  int tm, tn, split = 0;
  int m0, m1;  // rows of Y this tile may write: [m0, m1), at most BM
  const uint8_t* wq = a.wq;
  const float* sw = a.sw;
  if constexpr (GROUPED) {
    // Expert e owns the token slots offsets[e] / BM + e up to the next
    // expert's: at least ceil(count / BM) of them whatever the counts are, so
    // the host knows the number of slots without reading the offsets; the
    // slots past an expert's last row exit here.
    tn = work % a.tiles_n;
    const int slot = work / a.tiles_n;
    int e = -1;
    for (int e0 = 0; e0 < a.n_experts; e0 += 64) {
      bool mine = false;
      if (e0 + lane < a.n_experts)
        mine = min(max(a.offsets[e0 + lane], 0), a.M) / BM + e0 + lane <= slot;
      const unsigned long long b = __ballot(mine);
      if (b) e = e0 + 63 - __builtin_clzll(b);
      if (~b) break;
    }
    if (e < 0) return;
    e = __builtin_amdgcn_readfirstlane(e);
    const int lo = min(max(a.offsets[e], 0), a.M), hi = min(max(a.offsets[e + 1], 0), a.M);
    m0 = lo + (slot - lo / BM - e) * BM;
    m1 = min(m0 + BM, hi);
    if (m0 >= m1) return;
    wq += (long long)e * a.w_stride;
    sw += (long long)e * a.sw_stride;
  } else {
    split = work % a.split_k;
    work /= a.split_k;
    // bands of 8 token tiles, weight tiles inside a band in order: the ids an
    // XCD runs at one time form a near-square patch of tiles
    const int band = 8 * a.tiles_n;
    const int b0 = work / band * 8;
    const int h = min(8, a.tiles_m - b0);
    tn = work % band / h;
    tm = b0 + work % band % h;
    m0 = tm * BM;
    m1 = min(m0 + BM, a.M);
  }
  const int n0 = tn * BN;

  // ---- this wave's load addresses.  Row-major pieces are 8 rows x 128 bytes,
  // lane i holding row i / 8; the 16-byte chunk it loads is rotated by an
  // exclusive-or with the row, so that the 16 rows of an operand read fall
  // into different LDS banks.  Rows past the end repeat the last one (their
  // products are not stored).
  const int prow = lane >> 3, pchunk = (lane & 7) ^ prow;
  const int k_steps = a.G;
  const int ks0 = (int)((long long)k_steps * split / a.split_k);
  const int ks1 = (int)((long long)k_steps * (split + 1) / a.split_k);
  // a last step that K ends inside of: chunks past K re-read the last whole
  // one, and the token operand is masked after its LDS read
  const int tail_chunks = (a.K & 127) >> 4;
  const int tail_step = tail_chunks ? k_steps - 1 : -1;
  const int tail_adj = 16 * (min(pchunk, max(tail_chunks, 1) - 1) - pchunk);

  const uint8_t* px[T::PX];
  const uint8_t* pw[T::PW];
  auto x_row = [&](int i) -> long long {
    const int m = min(m0 + i, m1 - 1);
    if constexpr (GROUPED) {
      if (a.rows) return min(max(a.rows[m], 0), a.xrow_max);
    }
    return m;
  };
#pragma unroll
  for (int i = 0; i < T::PX; ++i) {
    const int p = min(wave + i * NW, T::X_BYTES / 1024 - 1);
    px[i] = a.xq + x_row(8 * p + prow) * a.ldq + 128 * (long long)ks0 + 16 * pchunk;
  }
#pragma unroll
  for (int i = 0; i < T::PW; ++i) {
    const int p = min(wave + i * NW, T::W_BYTES / 1024 - 1);
    if constexpr (PACKED) {
      // fragments of 16 rows x 128 bytes, 2 KiB per K-step, in lane order
      const int nb = min(n0 / 16 + p / 2, (a.N + 15) / 16 - 1);
      pw[i] = wq + ((long long)nb * k_steps + ks0) * 2048 + (p & 1) * 1024 + 16 * lane;
    } else {
      pw[i] = wq + min(n0 + 8 * p + prow, a.N - 1) * a.ldw + 128 * (long long)ks0 + 16 * pchunk;
    }
  }
  const unsigned lds0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;

  // Token scales: 16 bytes (four steps) per lane, token 32 p + lane / 2 of
  // piece p.  Near the end of a row the four are its last four (scale_at()
  // knows); a row of fewer than four goes in single words.
  const int G = a.G;
  const float* swt = sw + (long long)(n0 / 128) * G;
  const int sw_blocks = min((a.N + 127) / 128 - n0 / 128, (BN + 127) / 128);
  auto scale_start = [&](int g4) { return G >= 4 ? min(g4, G - 4) : g4; };
  auto issue_scales = [&](int c) {
    const unsigned base = lds0 + ST * T::STAGE + (c & 1) * T::SCALES;
    if (G >= 4) {
      for (int p = wave; p < T::SX_BYTES / 1024; p += NW)
        load_lds16(reinterpret_cast<const uint8_t*>(
                       a.sx + x_row(min(32 * p + (lane >> 1), BM - 1)) * G +
                       scale_start(8 * c + 4 * (lane & 1))),
                   base + p * 1024);
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

  auto issue = [&](int k, int stage) {
    const unsigned base = lds0 + stage * T::STAGE;
    const int adj = k == tail_step ? tail_adj : 0;
#pragma unroll
    for (int i = 0; i < T::PX; ++i) {
      const int p = min(wave + i * NW, T::X_BYTES / 1024 - 1);
      load_lds16(px[i] + adj, base + p * 1024);
      px[i] += 128;
    }
#pragma unroll
    for (int i = 0; i < T::PW; ++i) {
      const int p = min(wave + i * NW, T::W_BYTES / 1024 - 1);
      load_lds16(PACKED ? pw[i] : pw[i] + adj, base + T::X_BYTES + p * 1024);
      pw[i] += PACKED ? 2048 : 128;
    }
    // Scales of steps 8c .. 8c + 7 come with the first step that needs them:
    // a token's scales are consecutive in memory, so taking eight steps at
    // once fetches each cache line an eighth as often as one step would.
    if ((k & 7) == 0 || k == ks0) issue_scales(k >> 3);
  };

  v4f acc[NN][NM];
#pragma unroll
  for (int i = 0; i < NN; ++i)
#pragma unroll
    for (int j = 0; j < NM; ++j) acc[i][j] = v4f{0, 0, 0, 0};

#pragma unroll
  for (int s = 0; s < ST - 1; ++s) {
    // (steps past the end re-load the last one into a stage nobody reads)
    if (ks0 + s < ks1) issue(ks0 + s, s);
  }
  const int c0 = 16 * (q ^ (r & 7)), c1 = 16 * ((q + 4) ^ (r & 7));
  int stage = 0;
  for (int k = ks0; k < ks1; ++k) {
    // steps k .. k + ST - 2 are in flight, except near the end
    if (ST > 2 && k + ST - 2 < ks1)
      wait_stage<(ST - 2) * T::LOADS>();
    else
      wait_stage<0>();
    if (k + ST - 1 < ks1) issue(k + ST - 1, stage == 0 ? ST - 1 : stage - 1);
    uint8_t* xs = smem + stage * T::STAGE;
    if (k == tail_step) {
      // K ends inside this step: the tokens' chunks past it become zeros
      for (int c = threadIdx.x; c < BM * (8 - tail_chunks); c += T::THREADS) {
        const int row = c / (8 - tail_chunks), ch = tail_chunks + c % (8 - tail_chunks);
        *reinterpret_cast<v4i*>(xs + row * 128 + 16 * (ch ^ (row & 7))) = v4i{0, 0, 0, 0};
      }
      wait_stage<63>();
    }
    const uint8_t* ws = xs + T::X_BYTES + (wn * 16 * NN) * 128;
    xs += (wm * 16 * NM) * 128;
    const int g4 = scale_start(k & ~3);
    const uint8_t* ss = smem + ST * T::STAGE + ((k >> 3) & 1) * T::SCALES;
    const float swk =
        *reinterpret_cast<const float*>(ss + T::SX_BYTES + 32 * ((wn * 16 * NN) / 128) + 4 * (k & 7));
    ss += (wm * 16 * NM + r) * 32 + 16 * ((k >> 2) & 1) + 4 * (k - g4);
    v8i xf[NM];
    float sc[NM];
#pragma unroll
    for (int j = 0; j < NM; ++j) {
      const uint8_t* p = xs + (16 * j + r) * 128;
      const v4i lo = *reinterpret_cast<const v4i*>(p + c0);
      const v4i hi = *reinterpret_cast<const v4i*>(p + c1);
      xf[j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      sc[j] = *reinterpret_cast<const float*>(ss + 512 * j) * swk;
    }
#pragma unroll
    for (int i = 0; i < NN; ++i) {
      v4i lo, hi;
      if constexpr (PACKED) {
        lo = *reinterpret_cast<const v4i*>(ws + i * 2048 + 16 * lane);
        hi = *reinterpret_cast<const v4i*>(ws + i * 2048 + 1024 + 16 * lane);
      } else {
        const uint8_t* p = ws + (16 * i + r) * 128;
        lo = *reinterpret_cast<const v4i*>(p + c0);
        hi = *reinterpret_cast<const v4i*>(p + c1);
      }
      const v8i wf = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
      for (int j = 0; j < NM; ++j) {
        const v4f t = mfma_f8(wf, xf[j], v4f{0, 0, 0, 0});
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[i][j][u] = __builtin_fmaf(t[u], sc[j], acc[i][j][u]);
      }
    }
    stage = stage == ST - 1 ? 0 : stage + 1;
  }

  // ---- split-K: see the protocol of the small-M GEMM's shared tiles
  // (partials written through with agent scope, acknowledged, counted; the
  // last workgroup of the tile sums them in K order).
  if (!GROUPED && a.split_k > 1) {
    const int tile = work;
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
    int* flag = reinterpret_cast<int*>(smem);
    if (threadIdx.x == 0) {
      const unsigned inc = 256u / (unsigned)a.split_k;
      const unsigned prev = __hip_atomic_fetch_add(a.counters + (long long)tile * kCounterWords,
                                                   inc, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      *flag = ((prev + inc) & 255u) == 0u;
    }
    __syncthreads();
    if (!*flag) return;
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
#pragma unroll
    for (int i = 0; i < NN; ++i) {
#pragma unroll
      for (int j = 0; j < NM; ++j) acc[i][j] = v4f{0, 0, 0, 0};
      for (int s = 0; s < a.split_k; ++s)
#pragma unroll
        for (int j = 0; j < NM; ++j)
          acc[i][j] += __builtin_bit_cast(v4f, coherent_load16(prs, foff(s, i, j)));
    }
  }

  // ---- epilogue: lane (r, q) of tile (i, j) holds token 16 j + r, weight
  // rows 16 i + 4 q .. + 3
#pragma unroll
  for (int j = 0; j < NM; ++j) {
    const int m = m0 + (wm * NM + j) * 16 + r;
    if (m < m1) {
      uint16_t* yr = a.y + m * a.ldy;
#pragma unroll
      for (int i = 0; i < NN; ++i) {
        const int n = n0 + (wn * NN + i) * 16 + 4 * q;
        unsigned b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float f = acc[i][j][u];
          b[u] = f != f ? 0x7FC0u : (unsigned)bf16_rne(f);
        }
        if (a.vec_store && n + 4 <= a.N) {
          const v2u v = {b[0] | (b[1] << 16), b[2] | (b[3] << 16)};
          *reinterpret_cast<v2u*>(yr + n) = v;
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (n + u < a.N) yr[n + u] = (uint16_t)b[u];
        }
      }
    }
  }
}

typedef Tile<16, 128, 1, 4, 4> T0;
typedef Tile<32, 128, 1, 4, 4> T1;
typedef Tile<64, 128, 1, 4, 3> T2;
typedef Tile<128, 128, 2, 2, 2> T3;
typedef Tile<256, 256, 4, 2, 2> T4;

template <class T>
constexpr BlockTile describe() {
  return BlockTile{T::BM, T::BN, T::THREADS, T::LDS};
}
const BlockTile kTiles[kBlockTiles] = {describe<T0>(), describe<T1>(), describe<T2>(),
                                       describe<T3>(), describe<T4>()};

template <class T, bool GROUPED, bool PACKED>
hipError_t launch(const BlockGemmArgs& a, hipStream_t s) {
  // more than 64 KiB of LDS has to be asked for, once per kernel
  static const hipError_t lds = hipFuncSetAttribute(
      reinterpret_cast<const void*>(&block_gemm_kernel<T, GROUPED, PACKED>),
      hipFuncAttributeMaxDynamicSharedMemorySize, T::LDS);
  if (lds != hipSuccess) return lds;
  const unsigned wgs = (unsigned)((long long)a.tiles_m * a.tiles_n * a.split_k);
  hipLaunchKernelGGL((block_gemm_kernel<T, GROUPED, PACKED>), dim3(wgs), dim3(T::THREADS), T::LDS,
                     s, a);
  return hipGetLastError();
}

template <class T>
hipError_t launch_tile(bool grouped, bool packed, const BlockGemmArgs& a, hipStream_t s) {
  if (grouped) return packed ? launch<T, true, true>(a, s) : launch<T, true, false>(a, s);
  return packed ? launch<T, false, true>(a, s) : launch<T, false, false>(a, s);
}

}  // namespace

const BlockTile& block_tile(int tile) { return kTiles[tile]; }

hipError_t launch_block_gemm(int tile, bool grouped, bool packed, const BlockGemmArgs& a,
                             hipStream_t s) {
  switch (tile) {
    case 0: return launch_tile<T0>(grouped, packed, a, s);
    case 1: return launch_tile<T1>(grouped, packed, a, s);
    case 2: return launch_tile<T2>(grouped, packed, a, s);
    case 3: return launch_tile<T3>(grouped, packed, a, s);
    default: return launch_tile<T4>(grouped, packed, a, s);
  }
}

}  // namespace w8
