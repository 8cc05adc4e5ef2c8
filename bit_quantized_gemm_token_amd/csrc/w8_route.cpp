// C-ABI of the MoE operators around the grouped products: the routing, the
// combination of the experts' outputs and the whole layer of a few tokens.
// Argument checks first, then one launch or two, of the layer two or three; nothing
// here allocates, frees or synchronizes.
#include <algorithm>
#include <cstdint>
#include <string>

#include "w8_internal.hpp"
#include "w8_route.hpp"

using namespace w8;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

constexpr int kMaxRows = (1 << 22) - 1;  // (as the other operators for any token count)
constexpr int kMaxColumns = 1 << 20;     // of a combined row
constexpr int kMaxWidth = 1 << 16;       // D and I of the layer: 32-bit offsets of its partials
constexpr int kRouteBlocks = 1024;       // workgroups of the routing's first launch

w8_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws || have < need)
    return fail(W8_E_WORKSPACE, "workspace of " + std::to_string(need) + " bytes needed, got " +
                                    std::to_string(ws ? have : 0));
  if (!aligned(ws, 16)) return fail(W8_E_INVALID, "workspace must be 16-byte aligned");
  return W8_OK;
}

w8_status check_route(int T, int E, int topk) {
  if (T < 0 || T > kMaxRows)
    return fail(W8_E_INVALID, "T must be in [0, " + std::to_string(kMaxRows) + "], got " +
                                  std::to_string(T));
  if (E < 1 || E > kMaxExperts)
    return fail(W8_E_INVALID, "E must be in [1, " + std::to_string(kMaxExperts) + "], got " +
                                  std::to_string(E));
  if (topk < 1 || topk > kMaxTopk || topk > E)
    return fail(W8_E_INVALID, "topk must be in [1, " + std::to_string(std::min(kMaxTopk, E)) +
                                  "] (at most E), got " + std::to_string(topk));
  return W8_OK;
}

// One workgroup takes up to kRoutePass entries, unless its tokens come to several
// rounds of many choices, which cost more than the second launch (128 tokens of 300
// experts, top 2, 8 rounds 15.3 us, by two launches 9.0; 42 of 1000, top 6, 3 rounds
// 18.3 and 12.2; 24 of 300, top 8, 2 rounds 9.0 both; 64 of 300, top 1, 4 rounds 7.3
// and 8.0).  Otherwise a workgroup's pass is r rounds of its threads, which take
// longer by r - 1 times topk choices, and the second launch has fewer workgroups'
// counts to read: about 25 of them cost a choice's time (239 tokens of 256 experts,
// top 6: passes of 21 tokens 20.8 us, of 16 10.9; 261 of 8, top 1: of 128 11.7, of 16
// 7.3), with as many passes as keep the workgroups to kRouteBlocks.
void plan_route(RouteArgs* a) {
  const int lanes = route_lanes(a->T, a->E);
  const long long rounds = ceil_div((long long)a->T * lanes, kRouteWide);
  if ((long long)a->T * a->topk <= kRoutePass && (rounds - 1) * a->topk <= 8) {
    a->tokens = a->T;
  } else {
    const int round = kRouteThreads / lanes;
    int r = 1;
    while ((long long)(r + 1) * (r + 1) * round * a->topk * 25 <= a->T) ++r;
    a->tokens = std::min(r * round, kRouteMany / a->topk);
  }
  const long long passes = ceil_div(a->T, a->tokens);
  a->passes = (int)ceil_div(passes, kRouteBlocks);
  a->blocks = (int)ceil_div(passes, a->passes);
}

size_t route_bytes(const RouteArgs& a) {
  return a.blocks > 1 ? ws_counter_bytes(0) + (size_t)a.blocks * count_stride(a.E) * 4 : 0;
}

// The layer's workspace (byte offsets): the counter region that every
// operation keeps, then its arrays.
struct LayerWs {
  size_t h, hq, hs, part, total;
};
// Whether a launch of its own makes the codes of the hidden values, which otherwise
// every column tile makes again for its expert's tokens: by the values that a tile
// has to make, if the entries spread over the experts (32 tokens, 2 of 8 experts of
// 4096 x 14336, 114688 values: 270 us, 349 by the tiles; 4 of 16 of 4096 x 2048, 16384:
// 87 and 103; 2 of 16 of 2048 x 1024, 4096: 30.3 and 30.1; 16 tokens, 2 of 16 of 2048 x
// 2048, 4096: 41.6 and 40.7).
bool codes_apart(int n, int slots, int I) { return (long long)n * I >= 12288LL * slots; }

// Parts of I that workgroups of the layer's second kernel share where its columns
// and experts leave compute units without two of them (32 tokens, 2 of 8 experts of
// 1024 x 2048: in two 23.4 us, whole 27.3; 12 tokens, 4 of 16 of 256 x 4096, in four
// 21.0 and 28.6; 16 tokens, 2 of 60 of 384 x 4096, in two 37.7 and 42.9; 8 tokens, 2 of
// 16 of 1024 x 1024 15.6 and 15.1, which is why a part has 1024 columns at least).
int layer_splits(int slots, int D, int I) {
  const int tiles = (int)ceil_div(D, 64);
  int splits = 1;
  while (splits < 4 && (long long)tiles * slots * 2 * splits <= 512 && I >= 2048 * splits) splits *= 2;
  return splits;
}
// Bytes of an entry's codes: whole lines.
size_t coded_stride(int I) { return round256(I); }
LayerWs layer_ws(int T, int topk, int D, int I) {
  const size_t n = (size_t)T * topk;
  LayerWs w;
  w.h = ws_counter_bytes(0);
  w.hq = w.h + round256(n * I * 4);
  w.hs = w.hq + n * coded_stride(I);
  w.part = w.hs + round256(n * ceil_div(I, W8_GROUP) * 4);
  // (as many splits as one expert would take, and int8's scales: neither E nor the
  // format is known here)
  const int splits = layer_splits(1, D, I);
  w.total = w.part + round256(n * D * 4 * (splits > 1 ? splits + 1 : 1));
  return w;
}

w8_status check_layer(int fmt, int E, int T, int topk, int D, int I) {
  if (fmt < 0 || fmt > 2) return fail(W8_E_INVALID, "unknown format " + std::to_string(fmt));
  if (T < 0) return fail(W8_E_INVALID, "T must be >= 0");
  if (T > kLayerTokens)
    return fail(W8_E_UNSUPPORTED, "T=" + std::to_string(T) + " is above the few tokens the layer "
                                  "takes (" + std::to_string(kLayerTokens) + "); use the grouped "
                                  "products");
  if (E < 1 || E > kMaxExperts)
    return fail(W8_E_INVALID, "E must be in [1, " + std::to_string(kMaxExperts) + "], got " +
                                  std::to_string(E));
  if (topk < 1 || topk > kMaxTopk)
    return fail(W8_E_INVALID, "topk must be in [1, " + std::to_string(kMaxTopk) + "], got " +
                                  std::to_string(topk));
  const int unit = fmt == W8_BLOCK_FP8 ? W8_GROUP : 16;
  if (D < unit || D > kMaxWidth || D % unit || I < unit || I > kMaxWidth || I % unit)
    return fail(W8_E_INVALID, "D and I must be multiples of " + std::to_string(unit) + " up to " +
                                  std::to_string(kMaxWidth));
  return W8_OK;
}

// One of the layer's weights: [E, N, K] codes and their scales.
w8_status check_experts(int fmt, int E, int N, int K, const void* w, int64_t ldw,
                        int64_t w_stride, const float* s, int64_t s_stride) {
  if (!w || !s) return fail(W8_E_INVALID, "null device pointer");
  if (!aligned(w, 16) || !aligned(s, 4)) return fail(W8_E_INVALID, "misaligned weights or scales");
  if (ldw != 0 && (ldw < K || ldw % 16))
    return fail(W8_E_INVALID, "ldw must be >= K and a multiple of 16 (row-major) or 0 (packed)");
  const int64_t one = ldw == 0 ? (int64_t)packed_weight_bytes(fmt, N, K, 1)
                               : (int64_t)(N - 1) * ldw + K;
  // (of a single expert the strides are never used, and torch lets them be anything)
  if (E > 1 && (w_stride % 16 || w_stride < one))
    return fail(W8_E_INVALID, "the experts' stride must be a multiple of 16 that holds one's codes");
  const int64_t scales = fmt == W8_BLOCK_FP8 ? (int64_t)(N / W8_GROUP) * (K / W8_GROUP) : N;
  if (E > 1 && s_stride < scales)
    return fail(W8_E_INVALID, "the scales' stride must hold one expert's");
  return W8_OK;
}

// Up to 4 entries, and on short I up to 8 and up to 16 of one token's, take the
// second kernel for few entries, which reads an expert's weights for each entry that
// has chosen it and keeps one workgroup busy for 16 columns of all of them (2048 x
// 768, E experts: 1 token, 8 of 128 14.4 us, 16.1 by the other kernel; 2 tokens, 4 of
// 8 13.8 and 15.0; 8 tokens, 2 of 8 16.5 and 15.8; 1 token of 2048 x 4096: 2 of 8
// 25.1 and 27.4, 8 of 60 of 928 x 3360 31.0 and 23.3), with as many waves an entry as
// 16 leave, of 1024 columns of I at least (2 experts of 4096 x 4096: one wave 30.1 us,
// two 24.5, four 23.6; 4096 x 1024 12.6, 12.7 and 12.9).  0: the other kernel.
int layer_parts(int T, int topk, int I) {
  const int n = T * topk;
  if (n > (I > 1024 ? 4 : T == 1 ? 16 : 8)) return 0;
  int parts = 1;
  while (2 * parts * n <= 16 && I >= 2048 * parts) parts *= 2;
  return parts;
}

// Columns of I whose codes a workgroup of the layer's second kernel holds in
// LDS for each of `rows` rows, in 64 KiB less what the kernel needs itself:
// whole 128s.
int layer_chunk(int rows, int I) {
  const int per_row = 56 * 1024 / rows - 16;  // (codes, 16 bytes of padding, Block_FP8's scales)
  const int most = per_row * 32 / 33 / W8_GROUP * W8_GROUP;
  return std::min(most, (I + W8_GROUP - 1) / W8_GROUP * W8_GROUP);
}

}  // namespace

extern "C" {

w8_status w8_moe_route_workspace_size(int T, int E, int topk, size_t* bytes) {
  const w8_status st = check_route(T, E, topk);
  if (st) return st;
  if (!bytes) return fail(W8_E_INVALID, "null output pointer");
  RouteArgs a{};
  a.T = T;
  a.E = E;
  a.topk = topk;
  *bytes = 0;
  if (T) {
    plan_route(&a);
    *bytes = route_bytes(a);
  }
  return ok();
}

w8_status w8_moe_route(int T, int E, int topk, const void* logits, int64_t ldl, int logits_fp32,
                       int renormalize, float scale, int32_t* experts, float* weights,
                       int32_t* offsets, int32_t* rows, int32_t* slots, void* ws, size_t ws_bytes,
                       w8_stream stream) {
  w8_status st = check_route(T, E, topk);
  if (st) return st;
  if ((logits_fp32 != 0 && logits_fp32 != 1) || (renormalize != 0 && renormalize != 1))
    return fail(W8_E_INVALID, "logits_fp32 and renormalize must be 0 or 1");
  if (T == 0 && !offsets) return ok();
  if (T && (!logits || !experts || !weights)) return fail(W8_E_INVALID, "null device pointer");
  if (T && !offsets != !rows) return fail(W8_E_INVALID, "offsets, rows and slots go together");
  if (T && !offsets != !slots) return fail(W8_E_INVALID, "offsets, rows and slots go together");
  if (ldl < E) return fail(W8_E_INVALID, "ldl must be >= E");
  if (!aligned(logits, logits_fp32 ? 4 : 2) || !aligned(experts, 4) || !aligned(weights, 4) ||
      !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slots, 4))
    return fail(W8_E_INVALID, "every pointer must be aligned to its element type");
  RouteArgs a{logits, !logits_fp32, ldl, T, E, topk, renormalize, scale, experts, weights, offsets,
              rows, slots, 0, 0, 0, nullptr, 0};
  const int per = logits_fp32 ? 4 : 8;  // logits of 16 bytes
  a.wide = aligned(logits, 16) && ldl % per == 0 && E % per == 0;
  a.blocks = 1;  // (no tokens: the offsets alone)
  if (T) plan_route(&a);
  const size_t need = offsets ? route_bytes(a) : 0;
  if (need > 0) {
    st = check_workspace(ws, ws_bytes, need);
    if (st) return st;
    a.counts = reinterpret_cast<int*>(static_cast<char*>(ws) + ws_counter_bytes(0));
  }
  st = check_device();
  if (st) return st;
  const hipError_t e = launch_route(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(W8_E_HIP, hip_msg("moe_route launch", e));
  return ok();
}

w8_status w8_moe_combine(int T, int topk, int D, const void* y, int64_t ldy, int n_rows,
                         const float* weights, const int32_t* slots, const void* base, int64_t ldb,
                         void* out, int64_t ldo, w8_stream stream) {
  if (T < 0 || T > kMaxRows)
    return fail(W8_E_INVALID, "T must be in [0, " + std::to_string(kMaxRows) + "], got " +
                                  std::to_string(T));
  if (topk < 1 || topk > kMaxTopk)
    return fail(W8_E_INVALID, "topk must be in [1, " + std::to_string(kMaxTopk) + "], got " +
                                  std::to_string(topk));
  if (D < 1 || D > kMaxColumns) return fail(W8_E_INVALID, "D must be in [1, 2^20]");
  if (n_rows < 0) return fail(W8_E_INVALID, "n_rows must be >= 0");
  if (T == 0) return ok();
  if (!weights || !slots || !out || (n_rows && !y)) return fail(W8_E_INVALID, "null device pointer");
  if ((n_rows && ldy < D) || (base && ldb < D) || ldo < D)
    return fail(W8_E_INVALID, "leading dimensions must be >= D");
  if (!aligned(y, 2) || !aligned(base, 2) || !aligned(out, 2) || !aligned(weights, 4) ||
      !aligned(slots, 4))
    return fail(W8_E_INVALID, "every pointer must be aligned to its element type");
  // (a workgroup of 256 threads for at most 2048 columns of a token)
  if (T * ceil_div(D, 2048) * 256 > 0xFFFFFFFFLL)
    return fail(W8_E_INVALID, "the launch's threads exceed 2^32 - 1: split the call along T");
  const w8_status st = check_device();
  if (st) return st;
  const CombineArgs a{static_cast<const uint16_t*>(y), weights, slots,
                      static_cast<const uint16_t*>(base), static_cast<uint16_t*>(out), ldy, ldb,
                      ldo, T, D, topk, n_rows};
  const hipError_t e = launch_combine(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(W8_E_HIP, hip_msg("moe_combine launch", e));
  return ok();
}

w8_status w8_moe_layer_workspace_size(int T, int topk, int D, int I, size_t* bytes) {
  const w8_status st = check_layer(W8_FP8_DYNAMIC, 1, T, topk, D, I);
  if (st) return st;
  if (!bytes) return fail(W8_E_INVALID, "null output pointer");
  *bytes = T ? layer_ws(T, topk, D, I).total : 0;
  return ok();
}

w8_status w8_moe_layer(w8_fmt fmt_in, int E, int T, int topk, int D, int I, const void* xq,
                       int64_t ldq, const float* sx, const int32_t* experts, const float* weights,
                       const void* w1, int64_t ldw1, int64_t w1_stride, const float* s1,
                       int64_t s1_stride, const void* w2, int64_t ldw2, int64_t w2_stride,
                       const float* s2, int64_t s2_stride, const void* base, int64_t ldb, void* y,
                       int64_t ldy, void* ws, size_t ws_bytes, w8_stream stream) {
  const int fmt = raw_enum(fmt_in);
  w8_status st = check_layer(fmt, E, T, topk, D, I);
  if (st) return st;
  if (T == 0) return ok();
  if (!xq || !sx || !experts || !weights || !y) return fail(W8_E_INVALID, "null device pointer");
  if (!aligned(xq, 16) || ldq < D || ldq % 16)
    return fail(W8_E_INVALID, "xq must be 16-byte aligned with ldq >= D and ldq % 16 == 0");
  if (ldy < D || (base && ldb < D))
    return fail(W8_E_INVALID, "the output's and the base's leading dimensions must be >= D");
  if (!aligned(sx, 4) || !aligned(experts, 4) || !aligned(weights, 4) || !aligned(base, 2) ||
      !aligned(y, 2))
    return fail(W8_E_INVALID, "every pointer must be aligned to its element type");
  st = check_experts(fmt, E, 2 * I, D, w1, ldw1, w1_stride, s1, s1_stride);
  if (st) return st;
  st = check_experts(fmt, E, D, I, w2, ldw2, w2_stride, s2, s2_stride);
  if (st) return st;
  const LayerWs w = layer_ws(T, topk, D, I);
  st = check_workspace(ws, ws_bytes, w.total);
  if (st) return st;
  st = check_device();
  if (st) return st;
  char* p = static_cast<char*>(ws);
  MoeLayerArgs a{};
  a.xq = static_cast<const uint8_t*>(xq);
  a.sx = sx;
  a.experts = experts;
  a.weights = weights;
  a.w1 = static_cast<const uint8_t*>(w1);
  a.s1 = s1;
  a.w2 = static_cast<const uint8_t*>(w2);
  a.s2 = s2;
  a.base = static_cast<const uint16_t*>(base);
  a.ldb = ldb;
  a.y = static_cast<uint16_t*>(y);
  a.h = reinterpret_cast<float*>(p + w.h);
  a.part = reinterpret_cast<float*>(p + w.part);
  a.counters = static_cast<unsigned*>(ws);
  a.ldq = ldq;
  a.ldw1 = ldw1;
  a.ldw2 = ldw2;
  a.ldy = ldy;
  a.w1_stride = w1_stride;
  a.w2_stride = w2_stride;
  a.s1_stride = s1_stride;
  a.s2_stride = s2_stride;
  a.E = E;
  a.T = T;
  a.topk = topk;
  a.D = D;
  a.I = I;
  a.few = T * topk <= 64 && T * topk <= E;
  a.slots = std::min(E, T * topk);
  a.parts = layer_parts(T, topk, I);
  a.splits = a.parts ? 1 : layer_splits(a.slots, D, I);
  if (!a.parts && codes_apart(T * topk, a.slots, I)) {
    a.hq = reinterpret_cast<uint8_t*>(p + w.hq);
    a.hs = reinterpret_cast<float*>(p + w.hs);
    a.ldh = (long long)coded_stride(I);
  }
  const int each = a.parts ? a.parts : a.splits;
  a.chunk = layer_chunk(a.parts ? T * topk * a.parts : T,
                        each > 1 ? (I + each - 1) / each + W8_GROUP : I);
  const hipError_t e =
      launch_moe_layer(fmt, ldw1 == 0, ldw2 == 0, a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(W8_E_HIP, hip_msg("moe_layer launch", e));
  return ok();
}

}  // extern "C"
