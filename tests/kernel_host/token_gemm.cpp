// The token-scaled kernels of w8_block_gemm.hip on the CPU (hip/hip_runtime.h
// beside this file says how), behind one C function.
#include "w8_block_gemm.hip"

namespace w8 {
namespace {
__attribute__((aligned(1024))) uint8_t smem[160 * 1024];

template <class T, bool PACKED, int FMT>
void run_kernel(const BlockGemmArgs& a, unsigned wgs) {
  emu::m().lds = smem;
  emu::m().lds_bytes = T::LDS;
  for (unsigned b = 0; b < wgs && !emu::m().stop; ++b)
    emu::run_block(b, wgs, T::THREADS, [&] { block_gemm_kernel<T, PACKED, FMT>(a); });
}
template <class T, int FMT>
void run(bool packed, const BlockGemmArgs& a, unsigned wgs) {
  packed ? run_kernel<T, true, FMT>(a, wgs) : run_kernel<T, false, FMT>(a, wgs);
}
template <int FMT>
void run_tile(int tile, bool packed, const BlockGemmArgs& a, unsigned wgs) {
  switch (tile) {
    case kTile16x128: return run<T0, FMT>(packed, a, wgs);
    case kTile64x64: return run<T1, FMT>(packed, a, wgs);
    case kTile64x128: return run<T2, FMT>(packed, a, wgs);
    case kTile128x128: return run<T3, FMT>(packed, a, wgs);
    default: return run<T4, FMT>(packed, a, wgs);
  }
}
}  // namespace
}  // namespace w8

// The arguments of a launch, and the bytes behind its pointers.
struct EmuToken {
  int fmt, tile, packed, descending, late;
  int M, N, K, split_k, whole, parts, tiles_m, tiles_n;
  unsigned wgs;
  long long ldq, ldw, ldy;
  const uint8_t* xq;
  const float* sx;
  const uint8_t* wq;
  const float* sw;
  uint16_t* y;
  float* part;
  unsigned* counters;
  long long xq_bytes, sx_bytes, wq_bytes, sw_bytes, part_bytes;
};

// Number of faults; the first ones' text in emu_text().
extern "C" long long emu_token(const EmuToken* e) {
  using namespace w8;
  emu::Machine& g = emu::m();
  g.opt.descending = e->descending;
  g.opt.late = e->late;
  g.bad = g.loads = 0;
  g.stop = false;
  g.text.clear();
  g.ranges = {{"xq", e->xq, (size_t)e->xq_bytes},
              {"sx", (const uint8_t*)e->sx, (size_t)e->sx_bytes},
              {"wq", e->wq, (size_t)e->wq_bytes},
              {"sw", (const uint8_t*)e->sw, (size_t)e->sw_bytes},
              {"part", (const uint8_t*)e->part, (size_t)e->part_bytes}};
  BlockGemmArgs a{};
  a.xq = e->xq, a.sx = e->sx, a.wq = e->wq, a.sw = e->sw, a.y = e->y;
  a.part = e->part, a.counters = e->counters;
  a.ldq = e->ldq, a.ldw = e->ldw, a.ldy = e->ldy;
  a.M = e->M, a.N = e->N, a.K = e->K, a.G = (e->K + 127) / 128;
  a.split_k = e->split_k, a.whole = e->whole, a.parts = e->parts;
  a.tiles_m = e->tiles_m, a.tiles_n = e->tiles_n;
  if (e->fmt == W8A8_INT8)
    run_tile<W8A8_INT8>(e->tile, e->packed, a, e->wgs);
  else
    run_tile<FP8_DYNAMIC>(e->tile, e->packed, a, e->wgs);
  return g.bad;
}
extern "C" const char* emu_text() { return emu::m().text.c_str(); }
// The library's launcher: what it says to a tile.
extern "C" int emu_launch(int fmt, int tile, int packed) {
  const w8::BlockGemmArgs a{};
  return w8::launch_token_gemm(fmt, tile, 1, packed, a, nullptr);
}
