// MoE routing: each token's top-k experts and their weights from the router's
// logits, and the lists per expert that the grouped products take.
//
// The chosen are the k largest logits, ties to the lowest expert; -inf and NaN
// are never chosen.  The entries (token, choice) in order, sorted by expert
// with their order kept, are the lists: an entry's place is its expert's
// offset, plus the entries of that expert in front of it.  Those are counted
// within a pass of up to kRoutePass entries, over the passes of a workgroup and,
// in a second launch, over the workgroups: whole numbers in a fixed order, so
// the lists are the same every time.
//
// A row of logits is a few hundred bytes and stays in the registers of 16 or 64
// lanes as ordered keys.  Each choice is their maximum; a bf16 logit's key names its
// expert, an fp32 logit's is found again by a ballot, whose first lane holds the
// lowest.  So a token is a chain of topk reductions, and the chains of many tokens
// hide each other.
// Measured (medians of a trace): 8 tokens of 128 experts, top 8, 4.6 us in one
// launch, 32 tokens 5.4, all latency (1 token, 1 of 16 experts 3.1); 8192 tokens 5.8 us by
// the same chain (the bytes, 3.1 MB, take 1 us) and 6.9 us for the places, by the 256
// KiB of counts that each workgroup reads and the latency of reading, adding and
// writing one after the other.
#include "w8_block.hpp"
#include "w8_device.hpp"
#include "w8_route.hpp"
#include "w8_values.hpp"

namespace w8 {
namespace {

constexpr int kThreads = kRouteThreads;

// Over the L lanes (16 or 64) that share a token.
template <int L>
__device__ __forceinline__ unsigned lanes_umax(unsigned v) {
  return L == 16 ? seg16_umax(v) : wave_umax(v);
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  v += dpp_move<0xB1>(v);
  v += dpp_move<0x4E>(v);
  v += dpp_move<0x141>(v);
  v += dpp_move<0x140>(v);
  if (L == 16) return v;
  const int b = __builtin_bit_cast(int, v);
  const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
  const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
  const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
  const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
  return (r0 + r1) + (r2 + r3);
}

// Unsigned keys in the order of the logits; 0: never chosen (-inf, NaN).  The
// two zeros are one.  A bf16 logit's key leaves 16 bits free, which hold the
// expert, the lower the larger: such keys are all different.
__device__ __forceinline__ unsigned key_of(float l, bool there) {
  const unsigned u = l == 0.0f ? 0u : __float_as_uint(l);
  const unsigned key = u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
  return (there & (l > -__builtin_inff())) ? key : 0u;
}
template <bool HALF>
__device__ __forceinline__ float logit_of(unsigned key) {
  const unsigned u = key >> 31 ? key & 0x7FFFFFFFu : ~key;
  return __uint_as_float(HALF ? u & 0xFFFF0000u : u);
}

// exp(l - top), 1 at the top itself (where that is +inf too)
__device__ __forceinline__ float over_top(float l, float top) {
  return l == top ? 1.0f : expf(l - top);
}

// The place of each expert's first entry: an exclusive sum over count[0 .. E),
// by one workgroup; at[E] is the sum of all.  (at may be count.)
__device__ __forceinline__ void place_experts(const int* count, int* at, int E) {
  // the first wave, 16 experts a lane (E <= 1024)
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    const int per = (E + 63) / 64;
    int mine = 0;
    for (int i = 0; i < per; ++i) mine += lane * per + i < E ? count[lane * per + i] : 0;
    const int upto = wave_scan(mine);
    int sum = upto - mine;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e < E) {
        const int c = count[e];
        at[e] = sum;
        sum += c;
      }
    }
    if (lane == 63) at[E] = upto;
  }
}

// A lane's PER logits of a row from expert e0 on, as keys; wide: 16 bytes a load
// (aligned rows, whole pieces).  Loads past the row's end repeat its last ones,
// so that none waits for a condition.
template <int PER, typename Logit>
__device__ __forceinline__ void load_keys(const Logit* row, int e0, int E, bool wide,
                                          unsigned (&key)[PER]) {
  constexpr bool HALF = sizeof(Logit) == 2;
  constexpr int N = 16 / sizeof(Logit);
  static_assert(PER % N == 0, "whole loads");
  float l[PER];
  if (wide) {
    v4u v[PER / N];
#pragma unroll
    for (int c = 0; c < PER / N; ++c)
      v[c] = *reinterpret_cast<const v4u*>(row + min(e0 + c * N, E - N));
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const v4u& u = v[i / N];
      l[i] = HALF ? (i & 1 ? bf16_hi(u[i % N / 2]) : bf16_lo(u[i % N / 2]))
                  : __uint_as_float(u[HALF ? 0 : i % N]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const Logit v = row[min(e0 + i, E - 1)];
      if constexpr (HALF)
        l[i] = bf16_lo(v);
      else
        l[i] = v;
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    key[i] = key_of(l[i], e0 + i < E);
    if (HALF) key[i] = key[i] ? (key[i] & 0xFFFF0000u) | (0xFFFFu - (e0 + i)) : 0u;
  }
}

// L lanes take a token, PER logits each (E <= L * PER).  A choice is the largest
// key, over a lane's and then over the lanes; where keys can be equal, the first
// lane that holds it gives up its first.  Exponentials wait for the entries'
// turn, a thread each.
template <int THREADS, int L, int PER, typename Logit>
__global__ __launch_bounds__(THREADS) void route_kernel(RouteArgs a) {
  constexpr bool HALF = sizeof(Logit) == 2;
  __shared__ __align__(16) int ids[kRoutePass];
  __shared__ unsigned best_keys[kRoutePass];
  __shared__ float vals[kRoutePass];
  __shared__ float sums[kRoutePass];         // (not renormalized) of all experts, by token
  __shared__ int count[kMaxExperts + 1];     // entries of each expert in the passes so far
  const int sub = threadIdx.x % L, group = threadIdx.x / L;
  const bool lists = a.offsets != nullptr;
  if (a.T == 0) {  // (lists of nothing)
    for (int e = threadIdx.x; e <= a.E; e += THREADS) a.offsets[e] = 0;
    return;
  }
  for (int e = threadIdx.x; e < a.E; e += THREADS) count[e] = 0;
  for (int pass = 0; pass < a.passes; ++pass) {
    const long long t0 = ((long long)blockIdx.x * a.passes + pass) * a.tokens;
    if (t0 >= a.T) break;
    const int nt = (int)min((long long)a.tokens, a.T - t0);
    for (int t = group; t < nt; t += THREADS / L) {
      const Logit* row = static_cast<const Logit*>(a.logits) + (t0 + t) * a.ldl;
      unsigned key[PER];
      load_keys<PER>(row, sub * PER, a.E, a.wide, key);
      for (int j = 0; j < a.topk; ++j) {
        unsigned mine = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) mine = max(mine, key[i]);
        const unsigned best = lanes_umax<L>(mine);
        if (j == 0 && !a.renormalize) {
          const float top = logit_of<HALF>(best);
          float all = 0.0f;
#pragma unroll
          for (int i = 0; i < PER; ++i)
            all += key[i] ? over_top(logit_of<HALF>(key[i]), top) : 0.0f;
          all = lanes_sum<L>(all);
          if (sub == 0) sums[t] = all;
        }
        if constexpr (HALF) {
#pragma unroll
          for (int i = 0; i < PER; ++i) key[i] = key[i] == best ? 0u : key[i];
          if (sub == 0) best_keys[t * a.topk + j] = best;
        } else {
          // the first of the equals: lanes hold the experts in order
          unsigned long long at = __ballot(mine == best);
          if (L == 16) at = at >> (threadIdx.x & 48) & 0xFFFFu;
          const bool owner = sub == __builtin_ctzll(at);
          int e = PER;
#pragma unroll
          for (int i = PER - 1; i >= 0; --i) e = key[i] == best ? i : e;
          e = owner ? e : PER;
#pragma unroll
          for (int i = 0; i < PER; ++i) key[i] = i == e ? 0u : key[i];
          if (owner) {
            ids[t * a.topk + j] = best ? sub * PER + e : -1;
            best_keys[t * a.topk + j] = best;
          }
        }
      }
    }
    __syncthreads();
    // an entry a thread
    const int n = nt * a.topk, i = threadIdx.x;
    const int t = i / a.topk;
    const long long at = t0 * a.topk + i;
    int id = -1, rank = 0;
    if (i < n) {
      const unsigned best = best_keys[i];
      vals[i] = best ? over_top(logit_of<HALF>(best), logit_of<HALF>(best_keys[t * a.topk])) : 0.0f;
      if (HALF) ids[i] = best ? (int)(0xFFFFu - (best & 0xFFFFu)) : -1;
    }
    __syncthreads();
    if (i < n) {
      float sum = 0.0f;
      if (a.renormalize) {
        for (int j = 0; j < a.topk; ++j) sum += vals[t * a.topk + j];
      } else {
        sum = sums[t];
      }
      id = ids[i];
      a.experts[at] = id;
      a.weights[at] = id >= 0 ? a.scale * (vals[i] / sum) : 0.0f;
    }
    if (!lists) {
      __syncthreads();
      continue;
    }
    // An entry's rank is the number of entries of its expert in front of it: those
    // of its wave by comparing the expert's bits over the lanes, and what the waves
    // in front, which take their turns, have added to the expert's count.
    unsigned long long same = __ballot(id >= 0);
    for (int bit = 1; bit < a.E; bit *= 2) {
      const unsigned long long set = __ballot((id & bit) != 0);
      same &= id & bit ? set : ~set;
    }
    const int before =
        __builtin_amdgcn_mbcnt_hi((unsigned)(same >> 32),
                                  __builtin_amdgcn_mbcnt_lo((unsigned)same, 0u));
    for (int w = 0; w < n; w += 64) {
      // (the wave's lanes read a count before one of them adds to it: the fence keeps
      // the compiler from moving the write up)
      const bool turn = (int)threadIdx.x >> 6 == w >> 6 && id >= 0;
      if (turn) rank = count[id] + before;
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      if (turn && before == 0) count[id] = rank + __popcll(same);
      __syncthreads();
    }
    if (a.blocks > 1) {
      if (i < n) a.slots[at] = id >= 0 ? rank : -1;
      continue;
    }
    // (one workgroup has one pass)
    place_experts(count, count, a.E);
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += THREADS) a.offsets[e] = count[e];
    if (i < n) {
      a.slots[at] = id >= 0 ? count[id] + rank : -1;
      if (id >= 0) a.rows[count[id] + rank] = i / a.topk;
      if (i >= count[a.E]) a.rows[i] = 0;
    }
  }
  if (lists && a.blocks > 1) {
    __syncthreads();
    for (int e = threadIdx.x; e < count_stride(a.E); e += THREADS)
      a.counts[(long long)blockIdx.x * count_stride(a.E) + e] = e < a.E ? count[e] : 0;
  }
}

// The places of the entries of kSpan workgroups of route_kernel, from all
// workgroups' counts, which every workgroup here reads (64 KiB of L2 for each
// 128 of them and 128 experts): four experts a thread, the workgroups dealt to
// the threads.
constexpr int kPlaceThreads = 1024, kSpan = 8;

__global__ __launch_bounds__(kPlaceThreads) void place_kernel(RouteArgs a) {
  __shared__ int first[kMaxExperts + 4];        // of each expert
  __shared__ int before[kMaxExperts];           // entries of the workgroups in front of these
  __shared__ int next[kSpan][kMaxExperts];      // of each of these: its first entry's place
  const int b0 = blockIdx.x * kSpan, b1 = min(b0 + kSpan, a.blocks);
  const long long entries = (long long)a.T * a.topk;
  const long long each = (long long)a.passes * a.tokens * a.topk;
  const long long begin = b0 * each + threadIdx.x, end = min(b1 * each, entries);
  // (a thread's first entry, long before it is needed)
  int id = -1, rank = 0;
  if (begin < end) {
    id = a.experts[begin];
    rank = a.slots[begin];
  }
  const int stride = count_stride(a.E), quads = stride / 4;
  for (int e = threadIdx.x; e < stride; e += kPlaceThreads) {
    first[e] = 0;
    before[e] = 0;
  }
  __syncthreads();
  int width = 16;  // threads that take a workgroup's counts
  while (width < quads) width *= 2;
  const int q = threadIdx.x % width, step = kPlaceThreads / width;
  if (q < quads) {
    v4i all = {0, 0, 0, 0}, front = {0, 0, 0, 0};
#pragma unroll 8
    for (int b = threadIdx.x / width; b < a.blocks; b += step) {
      const v4i c = *reinterpret_cast<const v4i*>(a.counts + (long long)b * stride + 4 * q);
      all += c;
      if (b < b0) front += c;
      if (b >= b0 && b < b1) *reinterpret_cast<v4i*>(&next[b - b0][4 * q]) = c;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      atomicAdd(&first[4 * q + i], all[i]);
      atomicAdd(&before[4 * q + i], front[i]);
    }
  }
  __syncthreads();
  place_experts(first, first, a.E);
  __syncthreads();
  const int total = first[a.E];
  for (int e = threadIdx.x; e < a.E; e += kPlaceThreads) {
    int at = first[e] + before[e];
    for (int b = 0; b < b1 - b0; ++b) {
      const int c = next[b][e];
      next[b][e] = at;
      at += c;
    }
  }
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= a.E; e += kPlaceThreads) a.offsets[e] = first[e];
  __syncthreads();
  for (long long i = begin; i < end; i += kPlaceThreads) {
    if (i != begin) {
      id = a.experts[i];
      rank = a.slots[i];
    }
    if (id < 0) continue;
    const int slot = next[(int)(i / each) - b0][id] + rank;
    a.slots[i] = slot;
    a.rows[slot] = (int)(i / a.topk);
  }
  for (long long i = total + (long long)blockIdx.x * kPlaceThreads + threadIdx.x; i < entries;
       i += (long long)gridDim.x * kPlaceThreads)
    a.rows[i] = 0;
}

template <int THREADS, typename Logit>
auto pick(const RouteArgs& a) {
  if (route_lanes(a.T, a.E) == 16)
    return a.E <= 128 ? route_kernel<THREADS, 16, 8, Logit> : route_kernel<THREADS, 16, 16, Logit>;
  return a.E <= 512 ? route_kernel<THREADS, 64, 8, Logit> : route_kernel<THREADS, 64, 16, Logit>;
}
template <typename Logit>
hipError_t launch_first(const RouteArgs& a, hipStream_t s) {
  // (a single workgroup takes as many tokens at once as it can)
  const bool wide = a.blocks == 1 && (long long)a.T * route_lanes(a.T, a.E) > kThreads;
  return launch_kernel(wide ? pick<kRouteWide, Logit>(a) : pick<kThreads, Logit>(a),
                       dim3((unsigned)a.blocks), dim3(wide ? kRouteWide : kThreads), 0, s, a);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  const hipError_t e = a.bf16 ? launch_first<uint16_t>(a, s) : launch_first<float>(a, s);
  if (e != hipSuccess || !a.offsets || a.blocks == 1) return e;
  return launch_kernel(place_kernel, dim3((unsigned)((a.blocks + kSpan - 1) / kSpan)),
                       dim3(kPlaceThreads), 0, s, a);
}

}  // namespace w8
