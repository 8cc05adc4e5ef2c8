// The kernels of w8_block_gemm.hip on the CPU (hip/hip_runtime.h beside this
// file says how), behind one C function.
#include "w8_block_gemm.hip"

namespace w8 {
namespace {
__attribute__((aligned(1024))) uint8_t smem[160 * 1024];

template <class T, bool PACKED>
void run_kernel(bool grouped, const BlockGemmArgs& a, unsigned wgs) {
  emu::m().lds = smem;
  emu::m().lds_bytes = T::LDS;
  for (unsigned b = 0; b < wgs && !emu::m().stop; ++b)
    emu::run_block(b, wgs, T::THREADS, [&] {
      if constexpr (!std::is_same<T, T1>::value) {
        if (grouped) return grouped_gemm_kernel<T, PACKED>(a);
      }
      block_gemm_kernel<T, PACKED>(a);
    });
}
template <class T>
void run(bool grouped, bool packed, const BlockGemmArgs& a, unsigned wgs) {
  packed ? run_kernel<T, true>(grouped, a, wgs) : run_kernel<T, false>(grouped, a, wgs);
}
}  // namespace
}  // namespace w8

// The arguments of a launch, and the bytes behind its pointers.
struct EmuGemm {
  int tile, grouped, packed, descending, late;
  int M, N, K, split_k, whole, parts, tiles_m, tiles_n, n_experts, xrow_max;
  unsigned wgs;
  long long ldq, ldw, ldy, w_stride, sw_stride;
  const uint8_t* xq;
  const float* sx;
  const uint8_t* wq;
  const float* sw;
  uint16_t* y;
  float* part;
  unsigned* counters;
  const int* offsets;
  const int* rows;
  long long xq_bytes, sx_bytes, wq_bytes, sw_bytes, part_bytes;
};

// Number of faults; the first ones' text in emu_text().
extern "C" long long emu_gemm(const EmuGemm* e) {
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
  a.part = e->part, a.counters = e->counters, a.offsets = e->offsets, a.rows = e->rows;
  a.ldq = e->ldq, a.ldw = e->ldw, a.ldy = e->ldy;
  a.w_stride = e->w_stride, a.sw_stride = e->sw_stride;
  a.M = e->M, a.N = e->N, a.K = e->K, a.G = (e->K + 127) / 128;
  a.split_k = e->split_k, a.whole = e->whole, a.parts = e->parts;
  a.tiles_m = e->tiles_m, a.tiles_n = e->tiles_n;
  a.n_experts = e->n_experts, a.xrow_max = e->xrow_max;
  switch (e->tile) {
    case kTile16x128: run<T0>(e->grouped, e->packed, a, e->wgs); break;
    case kTile64x64: run<T1>(e->grouped, e->packed, a, e->wgs); break;
    case kTile64x128: run<T2>(e->grouped, e->packed, a, e->wgs); break;
    case kTile128x128: run<T3>(e->grouped, e->packed, a, e->wgs); break;
    default: run<T4>(e->grouped, e->packed, a, e->wgs);
  }
  return g.bad;
}
extern "C" const char* emu_text() { return emu::m().text.c_str(); }
extern "C" long long emu_loads() { return emu::m().loads; }
// The library's launchers: what they say to a tile.
extern "C" int emu_launch(int tile, int grouped, int packed) {
  const w8::BlockGemmArgs a{};
  return grouped ? w8::launch_grouped_gemm(tile, 1, packed, a, nullptr)
                 : w8::launch_block_gemm(tile, 1, packed, a, nullptr);
}
