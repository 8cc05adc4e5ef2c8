// Host-side declarations of the Block_FP8 operators for any token count: the
// argument blocks and launchers of the row operators (w8_rows.hip) and of the
// tiled GEMM (w8_block_gemm.hip), used by their C-ABI (w8_block.cpp).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace w8 {

// One kernel of one argument block, without the call configuration that the
// launch syntax pushes and pops (0.1 us of a call on the host).
template <class Args>
inline hipError_t launch_kernel(void (*kernel)(Args), dim3 grid, dim3 block, size_t lds,
                                hipStream_t s, Args args) {
  void* list[] = {&args};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, list, lds, s);
}

// ------------------------------------------------------------ row kernels --
struct BlockQuantArgs {
  const uint16_t* x;     // bf16 [M, K]
  const uint16_t* gate;  // bf16 [M, K], or null
  uint8_t* xq;           // codes [M, K]
  float* sx;             // [M, ceil(K/128)]
  long long ldx, ldg;    // elements
  long long ldq;         // bytes
  int K;
  unsigned G, groups;    // groups of a row and of all rows (below 2^31)
  unsigned magic;        // (set by the launcher) id / G as a multiplication
  int shift;
};
hipError_t launch_block_quantize(BlockQuantArgs a, hipStream_t s);

struct NormArgs {
  const uint16_t* y;         // bf16 [M, D]
  const void* residual;      // bf16 or fp32 [M, D]
  const uint16_t* gate;      // bf16 [D] (ldg 0) or [M, D], or null
  const uint16_t* post_w;    // bf16 [D], or null
  const uint16_t* w;         // bf16 [D]
  void* h;                   // [M, D] of the residual's type
  uint16_t* z;               // bf16 [M, D], or null
  uint8_t* zq;               // codes [M, D], or null
  float* sz;                 // [M, ceil(D/128)] with zq
  long long ldy, ldr, ldg, ldh, ldz;  // elements
  long long ldq;                      // bytes
  long long M;
  int D;
  int residual_fp32;
  float scale, eps;
};
constexpr int kNormMaxD = 32768;  // a row stays in one workgroup's registers
hipError_t launch_residual_norm(const NormArgs& a, hipStream_t s);

// ------------------------------------------------------------- tiled GEMM --
struct BlockGemmArgs {
  const uint8_t* xq;   // activation codes, row stride ldq bytes
  const float* sx;     // [rows, G]
  const uint8_t* wq;   // weight codes of expert 0
  const float* sw;     // [ceil(N/128), G] of expert 0
  uint16_t* y;         // bf16, row stride ldy elements
  float* part;         // split-K partials (workspace)
  unsigned* counters;  // split-K arrival counters (workspace)
  long long ldq, ldw, ldy;
  int M, N, K;
  int G;               // ceil(K / 128): scale groups and K-steps
  int split_k;         // power of two; 1 = whole K per workgroup
  int whole, parts;    // the largest tile: ids from `whole` on run in parts (2 or 4, 1: none do)
  int tiles_m;         // token tiles (grouped: slots, M / BM + min(E, M))
  int tiles_n;
  // grouped (per expert) products
  const int* offsets;      // [E + 1] (device)
  const int* rows;         // [M] token row of each entry (device), or null: entry i is row i
  long long w_stride;      // bytes between two experts' weights
  long long sw_stride;     // floats between two experts' scales
  int n_experts;
  int xrow_max;            // activation rows - 1
};

// A tile shape of the kernel: BM tokens x BN weight rows per workgroup.
struct BlockTile {
  int bm, bn, threads, lds_bytes;
};
// The tiles, by tokens x weight rows.  The largest runs a last, partial round
// in pieces and (grouped) short tiles at half height; kTile64x64 is not built
// for the grouped product.
enum BlockTileId { kTile16x128, kTile64x64, kTile64x128, kTile128x128, kTile256x256, kBlockTiles };
constexpr int kLargeTile = kTile256x256;
constexpr int kComputeUnits = 256;
// The largest tile takes a compute unit to itself.  The tiles of a last round
// that leaves at least half of the units idle run as two halves each, or where
// three quarters would idle as four quarters.
__host__ __device__ constexpr int last_round_parts(long long tiles) {
  const int rest = (int)(tiles % kComputeUnits);
  return rest == 0 || rest > kComputeUnits / 2 ? 1 : rest <= kComputeUnits / 4 ? 4 : 2;
}
constexpr int kGroupedPieces = 3 * kComputeUnits / 4;  // at most this many more than tiles
const BlockTile& block_tile(int tile);
// (hipErrorInvalidValue for a tile that is not built)
hipError_t launch_block_gemm(int tile, unsigned wgs, bool packed, const BlockGemmArgs& a,
                             hipStream_t s);
hipError_t launch_grouped_gemm(int tile, unsigned wgs, bool packed, const BlockGemmArgs& a,
                               hipStream_t s);

}  // namespace w8
