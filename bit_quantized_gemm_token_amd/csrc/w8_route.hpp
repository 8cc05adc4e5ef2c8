// Host-side declarations of the MoE operators around the grouped products: the
// routing (w8_route.hip), the combination of the experts' outputs (w8_rows.hip)
// and the whole layer of a few tokens (w8_moe_layer.hip), used by their C-ABI
// (w8_route.cpp).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace w8 {

constexpr int kMaxExperts = 1024;  // logits a wave holds; bits of the layer's expert set
constexpr int kMaxTopk = 32;
constexpr int kLayerTokens = 32;   // the small-M window

// ---------------------------------------------------------------- routing --
struct RouteArgs {
  const void* logits;  // bf16 or fp32 [T, E], row stride ldl elements
  int bf16;
  long long ldl;
  int T, E, topk;
  int renormalize;
  float scale;
  int* experts;    // [T, topk]
  float* weights;  // [T, topk]
  int* offsets;    // [E + 1], or null: no lists
  int* rows;       // [T * topk]
  int* slots;      // [T, topk]
  // T * topk entries in passes of `tokens` tokens (at most kRoutePass entries),
  // `passes` of them a workgroup; more than one workgroup: its experts' counts
  int tokens, passes, blocks;
  int* counts;  // [blocks, count_stride(E)] (workspace)
  int wide;     // rows load in 16-byte pieces
};
// Few entries are one pass of one workgroup (of kRouteWide threads where there are
// tokens for them); more go in passes of at most kRouteMany.
constexpr int kRoutePass = 256, kRouteMany = 128;
constexpr int kRouteThreads = 256, kRouteWide = 1024;
// Lanes that share a token: 16 hold up to 256 logits, 64 more.  Between 128 and
// 256 a choice takes 64 less time and 16 less work (256 experts, top 8: 1 token 5.4
// us and 7.1, 4096 tokens 17.7 and 14.5).
__host__ __device__ constexpr int route_lanes(int T, int E) {
  return E <= 128 || (E <= 256 && T > 16) ? 16 : 64;
}
__host__ __device__ constexpr int count_stride(int E) { return (E + 3) / 4 * 4; }
// One launch, or for more than one workgroup's entries two.
hipError_t launch_route(const RouteArgs& a, hipStream_t s);

// ------------------------------------------------------------ combination --
struct CombineArgs {
  const uint16_t* y;     // bf16 [n_rows, D]
  const float* weights;  // [T, topk]
  const int* slots;      // [T, topk]
  const uint16_t* base;  // bf16 [T, D], or null
  uint16_t* out;         // bf16 [T, D]
  long long ldy, ldb, ldo;
  int T, D, topk, n_rows;
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t s);

// ---------------------------------------------- the layer of a few tokens --
struct MoeLayerArgs {
  const uint8_t* xq;    // codes [T, D], row stride ldq bytes
  const float* sx;      // [T] or [T, D/128]
  const int* experts;   // [T, topk]
  const float* weights; // [T, topk]
  const uint8_t* w1;    // expert 0's gate rows, then up rows: [2 I, D]
  const float* s1;
  const uint8_t* w2;    // expert 0's [D, I]
  const float* s2;
  const uint16_t* base; // bf16 [T, D], or null
  uint16_t* y;          // bf16 [T, D]
  float* h;             // [T * topk, I] gated products (workspace)
  uint8_t* hq;          // codes of h [T * topk, I], row stride ldh bytes, or null: made where used
  float* hs;            // and their scales [T * topk] (Block_FP8: [T * topk, I / 128])
  long long ldh;
  float* part;          // [splits, T * topk, D] the experts' outputs (W8A8_INT8 in parts: the
                        // sums as int32, and behind them [T * topk, D] their scales)
  unsigned* counters;   // arrival counters
  long long ldq, ldw1, ldw2, ldb, ldy;  // bytes; base, y: elements
  long long w1_stride, w2_stride;       // bytes between experts
  long long s1_stride, s2_stride;       // floats
  int E, T, topk, D, I;
  int slots;            // of experts that a launch holds: each has tokens or ends at once
  int few;              // a slot is an entry (at most 64), else one of the experts with tokens
  int parts;            // > 0: few entries, so many waves each for the second product
  int splits;           // parts of I that workgroups of the second kernel share
  int chunk;            // of I that a workgroup of the second kernel (parts: a wave) keeps as codes
};
// Two launches, or three with hq.  packed1, packed2: the layouts of w1 and w2.
hipError_t launch_moe_layer(int fmt, bool packed1, bool packed2, const MoeLayerArgs& a,
                            hipStream_t s);

}  // namespace w8
