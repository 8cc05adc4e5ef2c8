// A GPU of one workgroup on the CPU, for tests: enough of the HIP device
// language and of gfx950's builtins to compile w8_block_gemm.hip with a host
// compiler and run its kernels thread by thread.
//
// Every thread of the workgroup is a fiber.  A fiber runs until it needs the
// other lanes of its wavefront (MFMA, readlane, ballot, DPP) or the other
// wavefronts (a barrier), or ends; the scheduler then takes the next fiber of
// the first wavefront that can run, in ascending or descending order.  So
// between two barriers one wavefront runs as far ahead of the others as the
// program lets it, which is the order that shows a missing barrier.
//
// Direct-to-LDS loads (w8_lds.hpp beside this file) are checked against the
// buffers the program registered, and land either at once or only when a wait
// asks for them: the two ends of what the memory may do.
#pragma once
#include <stddef.h>
#include <stdint.h>
#include <string.h>
#include <ucontext.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <deque>
#include <functional>
#include <memory>
#include <string>
#include <vector>

#define __host__
#define __device__
#define __global__
#define __shared__
#define __align__(n) __attribute__((aligned(n)))
#define __forceinline__ inline
#define __launch_bounds__(...)

typedef int hipError_t;
typedef void* hipStream_t;
constexpr hipError_t hipSuccess = 0, hipErrorInvalidValue = 1;
constexpr int hipFuncAttributeMaxDynamicSharedMemorySize = 8;
struct dim3 {
  unsigned x, y, z;
  dim3(unsigned x = 1, unsigned y = 1, unsigned z = 1) : x(x), y(y), z(z) {}
};
// (a launch through the library's own launchers is taken and does nothing)
inline hipError_t hipGetDevice(int* device) {
  *device = 0;
  return hipSuccess;
}
inline hipError_t hipFuncSetAttribute(const void*, int, int) { return hipSuccess; }
inline hipError_t hipLaunchKernel(const void*, dim3, dim3, void**, size_t, hipStream_t) {
  return hipSuccess;
}

namespace emu {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

struct Options {
  bool descending = false;  // wavefronts are tried from the last to the first
  bool late = false;        // direct-to-LDS loads land only when waited for
};

struct Range {
  const char* name;
  const uint8_t* p;
  size_t bytes;
};

struct Pending {
  unsigned lds;
  uint8_t data[16];
  int bytes;
};

struct Fiber {
  ucontext_t ctx;
  std::unique_ptr<char[]> stack;
  bool done = false, at_barrier = false, at_wave = false;
  std::deque<Pending> loads;
};

struct Machine {
  Options opt;
  std::vector<Range> ranges;
  std::vector<Fiber> fibers;
  ucontext_t home;
  int current = -1;
  unsigned block = 0, grid = 0;
  const std::function<void()>* body = nullptr;
  uint8_t* lds = nullptr;
  size_t lds_bytes = 0;
  long long bad = 0, loads = 0;
  bool stop = false;  // the program cannot go on (a fault too)
  std::string text;   // the first faults
  struct Wave {
    unsigned w[64][16];
    int op[64];
  };
  std::vector<Wave> in, out;
};
inline Machine& m() {
  static Machine machine;
  return machine;
}

inline void fault(const char* what) {
  Machine& g = m();
  if (g.bad++ < 4) g.text += std::string(what) + "\n";
}
inline void halt(const char* what) {
  fault(what);
  m().stop = true;
}
inline void fault(const char* what, const void* p, int bytes) {
  Machine& g = m();
  if (g.bad++ < 4) {
    const Range* nearest = nullptr;
    long long off = 0;
    for (const Range& r : g.ranges) {
      const long long o = (const uint8_t*)p - r.p;
      if (!nearest || std::llabs(o) < std::llabs(off)) nearest = &r, off = o;
    }
    char line[256];
    snprintf(line, sizeof line, "%s of %d bytes at %s + %lld (of %zu), block %u thread %d\n", what,
             bytes, nearest ? nearest->name : "?", off, nearest ? nearest->bytes : 0, g.block,
             g.current);
    g.text += line;
  }
}
inline bool inside(const void* p, int bytes) {
  for (const Range& r : m().ranges)
    if ((const uint8_t*)p >= r.p && (const uint8_t*)p + bytes <= r.p + r.bytes) return true;
  return false;
}

inline void yield() {
  Machine& g = m();
  swapcontext(&g.fibers[g.current].ctx, &g.home);
}
inline void barrier() {
  m().fibers[m().current].at_barrier = true;
  yield();
}

// One operation of a whole wavefront: every lane puts its words in, the last
// to arrive has them combined, every lane takes its result.
enum Op { kMfma = 1, kReadlane, kBallot, kDpp };
void combine(Machine::Wave& in, Machine::Wave& out);
inline unsigned* wave_op(int op, const void* words, size_t bytes) {
  Machine& g = m();
  const int w = g.current / 64, l = g.current % 64;
  memcpy(g.in[w].w[l], words, bytes);
  g.in[w].op[l] = op;
  g.fibers[g.current].at_wave = true;
  yield();
  return g.out[w].w[l];
}

inline float e4m3(uint8_t c) {
  static float table[256];
  static bool filled = false;
  if (!filled) {
    for (int i = 0; i < 256; ++i) {
      const int e = i >> 3 & 15, f = i & 7;
      const float v = e ? ldexpf(1 + f / 8.0f, e - 7) : ldexpf((float)f, -9);
      table[i] = e == 15 && f == 7 ? NAN : i & 128 ? -v : v;
    }
    filled = true;
  }
  return table[c];
}

inline void combine(Machine::Wave& in, Machine::Wave& out) {
  for (int l = 1; l < 64; ++l)
    if (in.op[l] != in.op[0]) return halt("lanes of one wavefront at different operations");
  if (in.op[0] == kMfma) {
    // lane l: row (first operand) or column (second) l % 16, one slice of K
    // by l / 16; result: column l % 16, rows 4 (l / 16) .. + 3
    static float a[16][128], b[16][128];
    for (int l = 0; l < 64; ++l)
      for (int i = 0; i < 32; ++i) {
        a[l % 16][l / 16 * 32 + i] = e4m3((uint8_t)(in.w[l][i / 4] >> 8 * (i % 4)));
        b[l % 16][l / 16 * 32 + i] = e4m3((uint8_t)(in.w[l][8 + i / 4] >> 8 * (i % 4)));
      }
    for (int l = 0; l < 64; ++l)
      for (int u = 0; u < 4; ++u) {
        const float *x = a[4 * (l / 16) + u], *y = b[l % 16];
        float s = 0;
        for (int k = 0; k < 128; ++k) s += x[k] * y[k];
        memcpy(&out.w[l][u], &s, 4);
      }
  } else if (in.op[0] == kReadlane) {
    for (int l = 0; l < 64; ++l) out.w[l][0] = in.w[in.w[l][1]][0];
  } else if (in.op[0] == kBallot) {
    unsigned long long v = 0;
    for (int l = 0; l < 64; ++l) v |= (unsigned long long)(in.w[l][0] != 0) << l;
    for (int l = 0; l < 64; ++l) memcpy(out.w[l], &v, 8);
  } else {  // DPP: words old, source, control, row mask
    for (int l = 0; l < 64; ++l) {
      const unsigned ctrl = in.w[l][2];
      int from = -1;
      if (ctrl > 0x110 && ctrl < 0x120) {  // row_shr
        const int n = ctrl - 0x110;
        if (l % 16 >= n) from = l - n;
      } else if (ctrl == 0x142) {  // row_bcast:15
        if (l >= 16) from = l / 16 * 16 - 1;
      } else if (ctrl == 0x143) {  // row_bcast:31
        if (l >= 32) from = 31;
      } else {
        return halt("a DPP control that is not known here");
      }
      const bool on = from >= 0 && (in.w[l][3] >> l / 16 & 1);
      out.w[l][0] = on ? in.w[from][1] : in.w[l][0];
    }
  }
}

inline v4f mfma(v8i a, v8i b, v4f c) {
  unsigned w[16];
  memcpy(w, &a, 32);
  memcpy(w + 8, &b, 32);
  v4f r;
  memcpy(&r, wave_op(kMfma, w, 64), 16);
  return r + c;
}
inline int readlane(int v, int lane) {
  const int w[2] = {v, lane};
  return (int)*wave_op(kReadlane, w, 8);
}
inline unsigned long long ballot(bool on) {
  const unsigned w = on;
  unsigned long long r;
  memcpy(&r, wave_op(kBallot, &w, 4), 8);
  return r;
}
inline int dpp(int old, int src, int ctrl, int row_mask) {
  const int w[4] = {old, src, ctrl, row_mask};
  return (int)*wave_op(kDpp, w, 16);
}

struct Rsrc {
  uint8_t* p;
  int bytes;
};
inline v4i rsrc_load(Rsrc r, int off) {
  v4i v{};
  if (off < 0 || off + 16 > r.bytes || !inside(r.p + off, 16))
    fault("load of a partial", r.p + off, 16);
  else
    memcpy(&v, r.p + off, 16);
  return v;
}
inline void rsrc_store(Rsrc r, int off, v4i v) {
  if (off < 0 || off + 16 > r.bytes || !inside(r.p + off, 16))
    fault("store of a partial", r.p + off, 16);
  else
    memcpy(r.p + off, &v, 16);
}

inline void entry() {
  (*m().body)();
  m().fibers[m().current].done = true;
  yield();
}

// One workgroup of `threads` threads running body().
inline void run_block(unsigned block, unsigned grid, int threads,
                      const std::function<void()>& body) {
  Machine& g = m();
  g.block = block;
  g.grid = grid;
  g.body = &body;
  constexpr size_t kStack = 256 * 1024;
  if ((int)g.fibers.size() < threads) g.fibers.resize(threads);
  const int waves = threads / 64;
  g.in.resize(waves);
  g.out.resize(waves);
  for (int i = 0; i < threads; ++i) {
    Fiber& f = g.fibers[i];
    if (!f.stack) f.stack.reset(new char[kStack]);
    f.done = f.at_barrier = f.at_wave = false;
    f.loads.clear();
    getcontext(&f.ctx);
    f.ctx.uc_stack.ss_sp = f.stack.get();
    f.ctx.uc_stack.ss_size = kStack;
    f.ctx.uc_link = nullptr;
    makecontext(&f.ctx, entry, 0);
  }
  memset(g.lds, 0x7F, g.lds_bytes);
  while (!g.stop) {
    bool ran = false;
    int alive = 0;
    for (int i = 0; i < waves && !ran; ++i) {
      const int w = g.opt.descending ? waves - 1 - i : i;
      int waiting = 0, live = 0;
      for (int l = 0; l < 64; ++l) {
        Fiber& f = g.fibers[64 * w + l];
        if (f.done) continue;
        ++live;
        if (f.at_wave) ++waiting;
        if (f.at_wave || f.at_barrier) continue;
        g.current = 64 * w + l;
        swapcontext(&g.home, &f.ctx);
        ran = true;
      }
      if (!ran && waiting) {
        if (waiting != 64) return halt("an operation of the whole wavefront with some lanes only");
        combine(g.in[w], g.out[w]);
        for (int l = 0; l < 64; ++l) g.fibers[64 * w + l].at_wave = false;
        ran = true;
      }
      alive += live;
    }
    if (ran) continue;
    if (!alive) break;
    for (int i = 0; i < threads; ++i) {  // every thread is at a barrier or has ended
      if (!g.fibers[i].done && !g.fibers[i].at_barrier) return halt("a deadlock");
      g.fibers[i].at_barrier = false;
    }
  }
  for (int i = 0; i < threads; ++i)
    if (!g.fibers[i].loads.empty()) return fault("a workgroup ends with loads in flight");
}

struct ThreadIdx {
  struct X {
    operator unsigned() const { return (unsigned)m().current; }
  } x;
};
struct BlockIdx {
  struct X {
    operator unsigned() const { return m().block; }
  } x;
};
struct GridDim {
  struct X {
    operator unsigned() const { return m().grid; }
  } x;
};
}  // namespace emu

static emu::ThreadIdx threadIdx;
static emu::BlockIdx blockIdx;
static emu::GridDim gridDim;

inline void __syncthreads() { emu::barrier(); }
inline unsigned long long __ballot(bool on) { return emu::ballot(on); }
inline unsigned __float_as_uint(float f) { return __builtin_bit_cast(unsigned, f); }
inline float __uint_as_float(unsigned u) { return __builtin_bit_cast(float, u); }
template <class A, class B>
inline auto min(A a, B b) { return a < b ? a : b; }
template <class A, class B>
inline auto max(A a, B b) { return a > b ? a : b; }
inline unsigned emu_fetch_add(unsigned* p, unsigned v) {
  const unsigned old = *p;
  *p += v;
  return old;
}

#define __HIP_MEMORY_SCOPE_AGENT 0
#define __hip_atomic_fetch_add(p, v, order, scope) emu_fetch_add(p, v)
#define __amdgpu_buffer_rsrc_t emu::Rsrc
#define __builtin_amdgcn_make_buffer_rsrc(p, stride, bytes, flags) \
  emu::Rsrc { (uint8_t*)(p), bytes }
#define __builtin_amdgcn_raw_buffer_load_b128(r, off, s, c) emu::rsrc_load(r, off)
#define __builtin_amdgcn_raw_buffer_store_b128(v, r, off, s, c) emu::rsrc_store(r, off, v)
#define __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, d, e, f, g, h, i) \
  emu::mfma(a, b, c)
#define __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, d, e, f) (c)
#define __builtin_amdgcn_cvt_pk_fp8_f32(a, b, old, hi) (old)
#define __builtin_amdgcn_readfirstlane(v) (v)
#define __builtin_amdgcn_readlane(v, l) emu::readlane(v, l)
#define __builtin_amdgcn_update_dpp(old, v, ctrl, rows, banks, bound) emu::dpp(old, v, ctrl, rows)
#define __builtin_amdgcn_sched_barrier(m) ((void)0)
#define __builtin_amdgcn_s_waitcnt(n) ((void)0)
