// C-ABI of the operators for any token count: Block_FP8's gated quantizer,
// residual norm, tiled GEMM and per-expert (grouped) GEMM, and the quantizer
// and tiled GEMM of the formats with one scale per token and output channel.
// Argument checks first, then one kernel launch each; nothing here allocates,
// frees or synchronizes.
#include <cstdint>
#include <string>

#include "w8_block.hpp"
#include "w8_internal.hpp"

using namespace w8;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int kMaxK = 1 << 22;
constexpr int kMaxN = 1 << 24;
// rows of one call: a launch holds at most 2^32 - 1 threads, and the row
// kernels take up to 1024 per row
constexpr int kMaxRows = (1 << 22) - 1;

constexpr int64_t kMaxStride = 1 << 23;

int groups_of(int K) { return (K + W8_GROUP - 1) / W8_GROUP; }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

w8_status check_rows(int M) {
  if (M < 0 || M > kMaxRows)
    return fail(W8_E_INVALID, "the number of rows must be in [0, " + std::to_string(kMaxRows) +
                                  "], got " + std::to_string(M));
  return W8_OK;
}

w8_status check_nk(int N, int K) {
  if (N < 1 || N > kMaxN) return fail(W8_E_INVALID, "N must be in [1, 2^24]");
  if (K < 16 || K > kMaxK || K % 16)
    return fail(W8_E_INVALID, "K must be a multiple of 16 in [16, 2^22]");
  return W8_OK;
}

// The formats with one scale per token and per output channel.
w8_status check_token_format(int fmt) {
  if (fmt != W8_FP8_DYNAMIC && fmt != W8_W8A8_INT8)
    return fail(W8_E_INVALID, "the format must be FP8_Dynamic or W8A8_INT8 (Block_FP8 has entry "
                              "points of its own), got " + std::to_string(fmt));
  return W8_OK;
}

// int8: sums of K products of any two codes, 2^14 at most each, stay in int32
constexpr int kMaxKInt8 = (1 << 17) - 16;

w8_status check_token_shape(int fmt, int M, int N, int K) {
  w8_status st = check_token_format(fmt);
  if (st) return st;
  st = check_rows(M);
  if (st) return st;
  st = check_nk(N, K);
  if (st) return st;
  if (fmt == W8_W8A8_INT8 && K > kMaxKInt8)
    return fail(W8_E_INVALID, "W8A8_INT8: K must be at most " + std::to_string(kMaxKInt8) +
                                  ", where any codes' sums stay in int32");
  return W8_OK;
}

w8_status check_ldq(int K, int64_t ldq) {
  if (ldq < K || ldq % 16)
    return fail(W8_E_INVALID, "ldq must be >= K and a multiple of 16");
  // (a tile's rows are addressed by 32-bit offsets from its first)
  if (ldq > kMaxStride) return fail(W8_E_INVALID, "ldq must be at most 2^23");
  return W8_OK;
}

w8_status check_layout(int packed) {
  if (packed != 0 && packed != 1)
    return fail(W8_E_INVALID, "weight layout must be 0 (row-major) or 1 (packed)");
  return W8_OK;
}

w8_status check_experts(int E, int T) {
  if (E < 1 || E > 65536) return fail(W8_E_INVALID, "E must be in [1, 65536]");
  if (T < 0) return fail(W8_E_INVALID, "T must be >= 0");
  return W8_OK;
}

// Operand checks shared by the dense and the grouped GEMM; *packed: the
// weight layout ldw names.
w8_status check_operands(int N, int K, const void* xq, int64_t ldq, const float* sx,
                         const void* wq, int64_t ldw, const float* sw, const void* y,
                         int64_t ldy, int* packed) {
  if (!xq || !sx || !wq || !sw || !y) return fail(W8_E_INVALID, "null device pointer");
  if (!aligned(xq, 16) || !aligned(wq, 16))
    return fail(W8_E_INVALID, "xq and wq must be 16-byte aligned");
  const w8_status st = check_ldq(K, ldq);
  if (st) return st;
  if (ldw != 0 && (ldw < K || ldw % 16))
    return fail(W8_E_INVALID, "ldw must be >= K and a multiple of 16 (row-major weights) or 0 "
                              "(packed; the K-segmented layouts are for the small-M GEMM)");
  if (ldw > kMaxStride) return fail(W8_E_INVALID, "ldw must be at most 2^23");
  *packed = ldw == 0;
  if (*packed && K % W8_GROUP) return fail(W8_E_INVALID, "packed weights need K % 128 == 0");
  if (ldy < N) return fail(W8_E_INVALID, "output leading dimension must be >= N");
  if (!aligned(sx, 4) || !aligned(sw, 4) || !aligned(y, 2))
    return fail(W8_E_INVALID, "misaligned scale or output pointer");
  return W8_OK;
}

// ------------------------------------------------------------ tile choice --
struct Plan {
  int tile, split_k;
  long long tiles_m, tiles_n;
  long long whole, wgs;  // the largest tile's whole tiles; workgroups
  int parts;             // the largest tile: pieces of each other tile
};

// Microseconds of a launch with `n` workgroups (output tiles times split_k) of
// `steps` K-steps each, fitted to 129 random shapes (20 <= M <= 8192, 256 <= N,
// K <= 8192) measured on every tile and every split_k of 1 .. 16: a step has
// one time with one workgroup on a compute unit and one with two; a round of
// workgroups costs its start and its output beside the steps; split K costs its
// hand-off and the partials' traffic.  On the shapes it was fitted to, the
// fastest of the estimates was within 1% of the fastest measured, on average (7%
// at worst); none were held back to check it on.  It orders the choices rather
// than tells times: for long runs of the largest tile, whose clock falls under
// power, it is 12 to 17% under what is measured (8192 x 5120 x 8192 244 us of
// 284 to 300).
//
// The token-scaled formats' steps are shorter by the additions of the groups'
// sums; their own costs were fitted the same way to 310 shapes (both formats,
// 14 to 8192 tokens), and on 104 others the choice was within 1.3% of the fastest
// measured on average, 17% at worst (by Block_FP8's costs 1.4%; 48 x 4608 x 7168
// 10.8 us on 64 x 128, K in four, where 64 x 64, K in two takes 9.5).
struct TileCost {
  int resident;         // workgroups of a compute unit
  double step1, step2;  // us a step, one or two of them resident
  double round;         // us a round beside the steps
};
struct Costs {
  TileCost tile[kBlockTiles];
  double launch;
  double half_step, quarter_step, piece_round;  // pieces of the largest tile
  double split, split_bytes;                    // K split: the hand-off, us a partial's byte
  double weight_bytes;                          // a us
};
constexpr Costs kBlockCosts = {
    {{2, 0.26, 0.50, 1.5}, {2, 0.23, 0.465, 2.0}, {2, 0.36, 0.725, 2.5}, {1, 0.47, 0.47, 3.15},
     {1, 1.305, 1.305, 7.4}},
    1.7, 0.89, 0.456, 3.3, 1.1, 0.38e-6, 4.5e6};
constexpr Costs kTokenCosts = {
    {{2, 0.208, 0.432, 1.15}, {2, 0.177, 0.418, 1.37}, {2, 0.319, 0.735, 1.85},
     {1, 0.439, 0.439, 2.73}, {1, 1.344, 1.344, 6.69}},
    1.67, 0.819, 0.433, 3.03, 1.33, 0.362e-6, 5.2e6};

double estimate(const Costs& costs, const Plan& p, int N, int K) {
  const TileCost& c = costs.tile[p.tile];
  const BlockTile& t = block_tile(p.tile);
  const int G = groups_of(K);
  const long long tiles = p.tiles_m * p.tiles_n, n = tiles * p.split_k;
  if (p.tile == kLargeTile)
    return costs.launch + (double)ceil_div(p.whole, kComputeUnits) * (G * c.step1 + c.round) +
           (p.whole < tiles
                ? G * (p.parts == 4 ? costs.quarter_step : costs.half_step) + costs.piece_round
                : 0);
  const double steps = (double)ceil_div(G, p.split_k);
  const long long cap = (long long)kComputeUnits * c.resident;
  double loop = (double)(n / cap) * (steps * c.step2 + c.round);
  if (n % cap) loop += steps * (n % cap <= kComputeUnits ? c.step1 : c.step2) + c.round;
  const double weights = (double)N * K / costs.weight_bytes;
  double us = costs.launch + (loop > weights ? loop : weights);
  if (p.split_k > 1) us += costs.split + costs.split_bytes * (double)n * t.bm * t.bn * 4;
  return us;
}

Plan plan_dense(int fmt, int M, int N, int K) {
  const Costs& costs = fmt == W8_BLOCK_FP8 ? kBlockCosts : kTokenCosts;
  Plan best{};
  double best_us = 0;
  for (int tile = 0; tile < kBlockTiles; ++tile) {
    Plan p{};
    p.tile = tile;
    const BlockTile& t = block_tile(tile);
    p.tiles_m = ceil_div(M, t.bm);
    p.tiles_n = ceil_div(N, t.bn);
    const long long tiles = p.tiles_m * p.tiles_n;
    p.whole = tiles;
    if (tile == kLargeTile) {
      p.parts = last_round_parts(tiles);
      if (p.parts > 1) p.whole = tiles - tiles % kComputeUnits;
    }
    // (a workgroup keeps two steps at least, and the arrival counters hold
    // kSplitKMaxTiles tiles)
    for (p.split_k = 1; p.split_k <= 16; p.split_k *= 2) {
      if (p.split_k > 1 && (tile == kLargeTile || tiles > kSplitKMaxTiles ||
                            groups_of(K) < 2 * p.split_k || tiles * p.split_k > 2 * kComputeUnits))
        break;
      p.wgs = tile == kLargeTile ? p.whole + p.parts * (tiles - p.whole) : tiles * p.split_k;
      const double us = estimate(costs, p, N, K);
      if (!best.wgs || us < best_us) {
        best = p;
        best_us = us;
      }
    }
  }
  return best;
}

// Up to W8_MAX_M tokens the small-M GEMM, whose waves stream the weights into
// registers, has the shorter start, and the tiles, whose loads do not wait for
// registers, the higher rate: the larger the weights and M, the better for the
// tiles (Block_FP8, on its untuned configurations: 1 x 2048 x 2048 4.1 us, tiles 5.2; 16 x
// 4096 x 4096 7.9 and 7.7; 24 x 4096 x 4096 9.7 and 7.8; 24 x 896 x 512 3.5 and
// 4.0; 1 x 4608 x 7168 12.5 and 9.8; 16 x 5120 x 8192 19.0 and 11.7).  Packed
// weights, which it reads in whole lines, move the border (1 x 5120 x 8192 10.8
// and 12.2; 8 x 5120 x 8192 12.4 and 11.7).  Block_FP8's needs whole groups.
bool use_small_m(int fmt, int M, int N, int K, bool packed) {
  if (M > W8_MAX_M) return false;
  const long long weights = (long long)N * K;
  // The token-scaled formats, both ways on 16 shapes of 0.5 M to 64 M weights and 14
  // token counts in both formats, with weights from memory and from the caches: this
  // rule is 0.0 to 3.1% and 0.2 to 0.7% over the faster of the two on average (by
  // layout and up to or above 16 tokens); Block_FP8's 1.9 to 6.2% and 0.2 to 3.2%;
  // the tiles alone 6 to 42% and 3 to 25%.  Around its borders, from memory, this
  // kernel and the tiles: 24 x 4096 x 2048 in int8 6.0 and 6.4 us, packed 5.3 and 6.4;
  // 24 x 1792 x 5120 9.4 and 7.6; 8 x 4608 x 7168 10.9 and 10.5, packed 9.3 and 10.3;
  // 16 x 5120 x 8192 packed 13.2 and 16.1.
  if (fmt != W8_BLOCK_FP8)
    return M > W8_MAX_M / 2 ? weights <= 8 << 20 : weights < 24 << 20 || packed;
  if (K % W8_GROUP) return false;
  if (M > W8_MAX_M / 2) return weights < 1 << 22;
  return weights < 24 << 20 || (packed && M < 8);
}

// The counts per expert are on the device, so their mean picks the tile: up to
// 8 rows the weights' bytes are all that counts and the smallest tile streams
// them best (128 experts of 1536 x 2048, 64 rows: 34.8 us, with the 64-row
// tile 36.4, the largest 49.0); up to 64 the 64-row tile (4096 rows of
// 2048 x 768: 51 us, 69 and 59); above, the largest, which runs short tiles at
// half height (32768 rows of 1536 x 2048: 164 us, 64-row tile 227, 128-row
// 214), unless it has few tiles for the compute units even in pieces (8 experts
// of 623 x 848, 5184 rows, 84 tiles: 12.9 us, 128-row tile 10.8; of 268 x 1216,
// 13320 rows, 120 tiles: 17.6 us and 22.4).  Where a smaller tile's
// workgroups all run at once still, its shorter steps win (64-row tile, one
// workgroup a compute unit, 16 experts of 260 x 448, 3942 rows: 6.4 us, 128-row
// 8.0; 16-row tile, two a unit where K is short, 60 experts of 512 x 512, 1588
// rows: 6.5, 64-row 7.1; of 420 x 1072, 805 rows: 11.6 and 9.9).
Plan plan_grouped(int E, int T, int N, int K, int64_t ldq, int n_rows) {
  const long long mean = n_rows / E, experts = n_rows < E ? n_rows : E;
  Plan p{};
  const auto take = [&](BlockTileId tile) {
    p.tile = tile;
    p.tiles_m = n_rows / block_tile(tile).bm + experts;
    p.tiles_n = ceil_div(N, block_tile(tile).bn);
  };
  // (half a tile an expert is what partial tiles add on average)
  const auto fits = [&](BlockTileId tile, int wgs) {
    return (n_rows / block_tile(tile).bm + experts / 2) * ceil_div(N, block_tile(tile).bn) <= wgs;
  };
  if (mean <= 8) {
    take(kTile16x128);
  } else if (mean <= 64) {
    take(kTile64x128);
  } else {
    take(kTile256x256);
    // (the largest tile addresses gathered rows by 32-bit offsets)
    if (p.tiles_m * p.tiles_n < 3 * kComputeUnits / 8 || (long long)T * ldq >= (1LL << 32))
      take(kTile128x128);
  }
  if (p.tile == kTile128x128 && fits(kTile64x128, kComputeUnits)) take(kTile64x128);
  const int run = groups_of(K) <= 6 ? 2 * kComputeUnits : kComputeUnits;
  if (p.tile == kTile64x128 && fits(kTile16x128, run)) take(kTile16x128);
  p.split_k = p.parts = 1;
  p.whole = p.wgs = p.tiles_m * p.tiles_n;
  if (p.tile == kLargeTile) p.wgs += kGroupedPieces;
  return p;
}

size_t plan_bytes(const Plan& p) {
  if (p.split_k == 1) return 0;
  const BlockTile& t = block_tile(p.tile);
  return ws_counter_bytes(0) + (size_t)(p.tiles_m * p.tiles_n) * p.split_k * t.bm * t.bn * 4;
}

w8_block_plan describe(const Plan& p) {
  const BlockTile& t = block_tile(p.tile);
  return {t.bm, t.bn, p.split_k, p.tile == kLargeTile ? p.parts : 1, p.wgs};
}

w8_status check_grid(const Plan& p) {
  const long long threads = p.wgs * block_tile(p.tile).threads;
  if (threads > 0xFFFFFFFFLL)
    return fail(W8_E_INVALID, "the launch's threads exceed 2^32 - 1: split the call along M or N");
  return W8_OK;
}

// Arguments of a quantizer (M == 0 needs no buffers).
w8_status check_quantize(int M, int K, const void* x, int64_t ldx, const void* gate, int64_t ldg,
                         const void* xq, int64_t ldq, const float* sx) {
  const w8_status st = check_rows(M);
  if (st) return st;
  if (K < 8 || K > kMaxK || K % 8)
    return fail(W8_E_INVALID, "K must be a multiple of 8 in [8, 2^22]");
  if (M == 0) return W8_OK;
  if (!x || !xq || !sx) return fail(W8_E_INVALID, "null device pointer");
  if (!aligned(x, 16) || ldx % 8 || ldx < K)
    return fail(W8_E_INVALID, "x must be 16-byte aligned with ldx >= K and ldx % 8 == 0");
  if (gate && (!aligned(gate, 16) || ldg % 8 || ldg < K))
    return fail(W8_E_INVALID, "gate must be 16-byte aligned with ldg >= K and ldg % 8 == 0");
  if (!aligned(xq, 8) || ldq % 8 || ldq < K)
    return fail(W8_E_INVALID, "xq must be 8-byte aligned with ldq >= K and ldq % 8 == 0");
  if (!aligned(sx, 4)) return fail(W8_E_INVALID, "sx must be 4-byte aligned");
  return W8_OK;
}

// The dense GEMM of any format, its shape checked and M > 0.
w8_status dense_gemm(int fmt, int M, int N, int K, const void* xq, int64_t ldq, const float* sx,
                     const void* wq, int64_t ldw, const float* sw, void* y, int64_t ldy, void* ws,
                     size_t ws_bytes, w8_stream stream) {
  int packed = 0;
  w8_status st = check_operands(N, K, xq, ldq, sx, wq, ldw, sw, y, ldy, &packed);
  if (st) return st;
  if (use_small_m(fmt, M, N, K, packed))
    return w8_gemm_w8a8((w8_fmt)fmt, M, N, K, xq, ldq, sx, wq, ldw, sw, y, ldy, nullptr, ws,
                        ws_bytes, stream);
  const Plan p = plan_dense(fmt, M, N, K);
  const size_t need = plan_bytes(p);
  if (need > 0) {
    if (!ws || ws_bytes < need)
      return fail(W8_E_WORKSPACE, "workspace of " + std::to_string(need) + " bytes needed, got " +
                                      std::to_string(ws ? ws_bytes : 0));
    if (!aligned(ws, 16)) return fail(W8_E_INVALID, "workspace must be 16-byte aligned");
  }
  st = check_grid(p);
  if (st) return st;
  st = check_device();
  if (st) return st;
  BlockGemmArgs a{};
  a.xq = static_cast<const uint8_t*>(xq);
  a.sx = sx;
  a.wq = static_cast<const uint8_t*>(wq);
  a.sw = sw;
  a.y = static_cast<uint16_t*>(y);
  if (need > 0) {
    a.counters = static_cast<unsigned*>(ws);
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + ws_counter_bytes(0));
  }
  a.ldq = ldq;
  a.ldw = ldw;
  a.ldy = ldy;
  a.M = M;
  a.N = N;
  a.K = K;
  a.G = groups_of(K);
  a.split_k = p.split_k;
  a.whole = (int)p.whole;
  a.parts = p.parts;
  a.tiles_m = (int)p.tiles_m;
  a.tiles_n = (int)p.tiles_n;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = fmt == W8_BLOCK_FP8
                           ? launch_block_gemm(p.tile, (unsigned)p.wgs, packed, a, s)
                           : launch_token_gemm(fmt, p.tile, (unsigned)p.wgs, packed, a, s);
  if (e != hipSuccess) return fail(W8_E_HIP, hip_msg("tiled GEMM launch", e));
  return ok();
}

}  // namespace

extern "C" {

w8_status w8_block_quantize(int M, int K, const void* x, int64_t ldx, const void* gate,
                            int64_t ldg, void* xq, int64_t ldq, float* sx, w8_stream stream) {
  w8_status st = check_quantize(M, K, x, ldx, gate, ldg, xq, ldq, sx);
  if (st) return st;
  if ((long long)M * groups_of(K) >= (1LL << 31))
    return fail(W8_E_INVALID, "the groups (M x ceil(K / 128)) must be fewer than 2^31");
  if (M == 0) return ok();
  st = check_device();
  if (st) return st;
  BlockQuantArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(gate),
                   static_cast<uint8_t*>(xq), sx, ldx, ldg, ldq, K, (unsigned)groups_of(K),
                   (unsigned)M * (unsigned)groups_of(K), 0, 0};
  const hipError_t e = launch_block_quantize(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(W8_E_HIP, hip_msg("block_quantize launch", e));
  return ok();
}

w8_status w8_residual_norm(int M, int D, const void* y, int64_t ldy, const void* residual,
                           int64_t ldr, int residual_fp32, const void* post_weight,
                           const void* gate, int64_t ldg, float scale, const void* weight,
                           float eps, void* h, int64_t ldh, void* z, int64_t ldz, void* zq,
                           int64_t ldq, float* sz, w8_stream stream) {
  w8_status st = check_rows(M);
  if (st) return st;
  if (D < 1) return fail(W8_E_INVALID, "D must be positive");
  if (D > kNormMaxD)
    return fail(W8_E_UNSUPPORTED, "D=" + std::to_string(D) + " is above the row length that the "
                                  "norm keeps in registers (" + std::to_string(kNormMaxD) +
                                  "); use another backend");
  if (residual_fp32 != 0 && residual_fp32 != 1)
    return fail(W8_E_INVALID, "residual_fp32 must be 0 or 1");
  if (!(eps >= 0.0f)) return fail(W8_E_INVALID, "eps must be >= 0");
  if (M == 0) return ok();
  if (!y || !residual || !weight || !h) return fail(W8_E_INVALID, "null device pointer");
  if (!z && !zq) return fail(W8_E_INVALID, "at least one of z and zq must be given");
  if (zq && !sz) return fail(W8_E_INVALID, "zq needs sz");
  if (ldy < D || ldr < D || ldh < D || (gate && ldg != 0 && ldg < D) || (z && ldz < D) ||
      (zq && ldq < D))
    return fail(W8_E_INVALID, "leading dimensions must be >= D (gate: or 0, one row for all)");
  const size_t ra = residual_fp32 ? 4 : 2;
  if (!aligned(y, 2) || !aligned(residual, ra) || !aligned(h, ra) || !aligned(weight, 2) ||
      !aligned(post_weight, 2) || !aligned(gate, 2) || !aligned(z, 2) || !aligned(sz, 4))
    return fail(W8_E_INVALID, "every pointer must be aligned to its element type");
  st = check_device();
  if (st) return st;
  NormArgs a{static_cast<const uint16_t*>(y), residual, static_cast<const uint16_t*>(gate),
             static_cast<const uint16_t*>(post_weight), static_cast<const uint16_t*>(weight), h,
             static_cast<uint16_t*>(z), static_cast<uint8_t*>(zq), sz, ldy, ldr, ldg, ldh, ldz,
             ldq, M, D, residual_fp32, scale, eps};
  const hipError_t e = launch_residual_norm(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(W8_E_HIP, hip_msg("residual_norm launch", e));
  return ok();
}

w8_status w8_block_gemm_workspace_size(int M, int N, int K, int packed, size_t* bytes) {
  w8_status st = check_rows(M);
  if (st) return st;
  st = check_nk(N, K);
  if (st) return st;
  st = check_layout(packed);
  if (st) return st;
  if (!bytes) return fail(W8_E_INVALID, "null output pointer");
  if (M && use_small_m(W8_BLOCK_FP8, M, N, K, packed))
    return w8_workspace_size(W8_BLOCK_FP8, W8_OP_GEMM, M, N, K, packed, nullptr, bytes);
  *bytes = M ? plan_bytes(plan_dense(W8_BLOCK_FP8, M, N, K)) : 0;
  return ok();
}

w8_status w8_block_gemm_plan(int M, int N, int K, int packed, w8_block_plan* plan) {
  w8_status st = check_rows(M);
  if (st) return st;
  st = check_nk(N, K);
  if (st) return st;
  st = check_layout(packed);
  if (st) return st;
  if (packed && K % W8_GROUP) return fail(W8_E_INVALID, "packed weights need K % 128 == 0");
  if (!plan) return fail(W8_E_INVALID, "null output pointer");
  *plan = w8_block_plan{0, 0, 1, 1, 0};
  if (M && !use_small_m(W8_BLOCK_FP8, M, N, K, packed)) *plan = describe(plan_dense(W8_BLOCK_FP8, M, N, K));
  return ok();
}

w8_status w8_block_gemm(int M, int N, int K, const void* xq, int64_t ldq, const float* sx,
                        const void* wq, int64_t ldw, const float* sw, void* y, int64_t ldy,
                        void* ws, size_t ws_bytes, w8_stream stream) {
  w8_status st = check_rows(M);
  if (st) return st;
  st = check_nk(N, K);
  if (st) return st;
  if (M == 0) return ok();
  return dense_gemm(W8_BLOCK_FP8, M, N, K, xq, ldq, sx, wq, ldw, sw, y, ldy, ws, ws_bytes, stream);
}

w8_status w8_token_gemm_workspace_size(w8_fmt fmt_in, int M, int N, int K, int packed,
                                       size_t* bytes) {
  const int fmt = raw_enum(fmt_in);
  w8_status st = check_token_shape(fmt, M, N, K);
  if (st) return st;
  st = check_layout(packed);
  if (st) return st;
  if (!bytes) return fail(W8_E_INVALID, "null output pointer");
  if (M && use_small_m(fmt, M, N, K, packed))
    return w8_workspace_size((w8_fmt)fmt, W8_OP_GEMM, M, N, K, packed, nullptr, bytes);
  *bytes = M ? plan_bytes(plan_dense(fmt, M, N, K)) : 0;
  return ok();
}

w8_status w8_token_gemm_plan(w8_fmt fmt_in, int M, int N, int K, int packed, w8_block_plan* plan) {
  const int fmt = raw_enum(fmt_in);
  w8_status st = check_token_shape(fmt, M, N, K);
  if (st) return st;
  st = check_layout(packed);
  if (st) return st;
  if (packed && K % W8_GROUP) return fail(W8_E_INVALID, "packed weights need K % 128 == 0");
  if (!plan) return fail(W8_E_INVALID, "null output pointer");
  *plan = w8_block_plan{0, 0, 1, 1, 0};
  if (M && !use_small_m(fmt, M, N, K, packed)) *plan = describe(plan_dense(fmt, M, N, K));
  return ok();
}

w8_status w8_token_gemm(w8_fmt fmt_in, int M, int N, int K, const void* xq, int64_t ldq,
                        const float* sx, const void* wq, int64_t ldw, const float* sw, void* y,
                        int64_t ldy, void* ws, size_t ws_bytes, w8_stream stream) {
  const int fmt = raw_enum(fmt_in);
  const w8_status st = check_token_shape(fmt, M, N, K);
  if (st) return st;
  if (M == 0) return ok();
  return dense_gemm(fmt, M, N, K, xq, ldq, sx, wq, ldw, sw, y, ldy, ws, ws_bytes, stream);
}

w8_status w8_token_quantize(w8_fmt fmt_in, int M, int K, const void* x, int64_t ldx,
                            const void* gate, int64_t ldg, int reciprocal, void* xq, int64_t ldq,
                            float* sx, w8_stream stream) {
  const int fmt = raw_enum(fmt_in);
  w8_status st = check_token_format(fmt);
  if (st) return st;
  if (reciprocal != 0 && reciprocal != 1) return fail(W8_E_INVALID, "reciprocal must be 0 or 1");
  st = check_quantize(M, K, x, ldx, gate, ldg, xq, ldq, sx);
  if (st) return st;
  if (M == 0) return ok();
  st = check_device();
  if (st) return st;
  const TokenQuantArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(gate),
                         static_cast<uint8_t*>(xq), sx, ldx, ldg, ldq, M, K, reciprocal};
  const hipError_t e = launch_token_quantize(fmt, a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(W8_E_HIP, hip_msg("token_quantize launch", e));
  return ok();
}

w8_status w8_grouped_gemm_plan(int E, int T, int N, int K, int64_t ldq, int n_rows,
                               w8_block_plan* plan) {
  w8_status st = check_rows(n_rows);
  if (st) return st;
  st = check_nk(N, K);
  if (st) return st;
  st = check_experts(E, T);
  if (st) return st;
  st = check_ldq(K, ldq);
  if (st) return st;
  if (!plan) return fail(W8_E_INVALID, "null output pointer");
  *plan = w8_block_plan{0, 0, 1, 1, 0};
  if (n_rows) *plan = describe(plan_grouped(E, T, N, K, ldq, n_rows));
  return ok();
}

w8_status w8_grouped_gemm(int E, int T, int N, int K, const void* xq, int64_t ldq,
                          const float* sx, const int32_t* offsets, const int32_t* rows,
                          int n_rows, const void* wq, int64_t ldw, int64_t w_stride,
                          const float* sw, int64_t sw_stride, void* y, int64_t ldy,
                          w8_stream stream) {
  w8_status st = check_rows(n_rows);
  if (st) return st;
  st = check_nk(N, K);
  if (st) return st;
  st = check_experts(E, T);
  if (st) return st;
  if (n_rows == 0) return ok();
  if (T < 1) return fail(W8_E_INVALID, "routed entries need at least one token row");
  if (!offsets) return fail(W8_E_INVALID, "null device pointer");
  if (!rows && T < n_rows)
    return fail(W8_E_INVALID, "without a row list entry i is row i: T must be >= n_rows");
  int packed = 0;
  st = check_operands(N, K, xq, ldq, sx, wq, ldw, sw, y, ldy, &packed);
  if (st) return st;
  if (!aligned(offsets, 4) || !aligned(rows, 4))
    return fail(W8_E_INVALID, "offsets and rows must be 4-byte aligned");
  const int64_t one = packed ? (int64_t)packed_weight_bytes(W8_BLOCK_FP8, N, K, 1)
                             : (int64_t)(N - 1) * ldw + K;
  if (w_stride % 16 || (E > 1 && w_stride < one))
    return fail(W8_E_INVALID, "w_stride must be a multiple of 16 that holds one expert's codes");
  if (E > 1 && sw_stride < (int64_t)groups_of(N) * groups_of(K))
    return fail(W8_E_INVALID, "sw_stride must hold one expert's scales");
  const Plan p = plan_grouped(E, T, N, K, ldq, n_rows);
  st = check_grid(p);
  if (st) return st;
  st = check_device();
  if (st) return st;
  BlockGemmArgs a{};
  a.xq = static_cast<const uint8_t*>(xq);
  a.sx = sx;
  a.wq = static_cast<const uint8_t*>(wq);
  a.sw = sw;
  a.y = static_cast<uint16_t*>(y);
  a.ldq = ldq;
  a.ldw = ldw;
  a.ldy = ldy;
  a.M = n_rows;
  a.N = N;
  a.K = K;
  a.G = groups_of(K);
  a.split_k = 1;
  a.tiles_m = (int)p.tiles_m;
  a.tiles_n = (int)p.tiles_n;
  a.offsets = offsets;
  a.rows = rows;
  a.w_stride = w_stride;
  a.sw_stride = sw_stride;
  a.n_experts = E;
  a.xrow_max = T - 1;
  const hipError_t e =
      launch_grouped_gemm(p.tile, (unsigned)p.wgs, packed, a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(W8_E_HIP, hip_msg("grouped_gemm launch", e));
  return ok();
}

}  // extern "C"
