// The direct-to-LDS loads and the waits of csrc/w8_lds.hpp on the CPU: every
// source address is checked, and the bytes land at once or, in order, when a
// wait asks for them.
#pragma once
#include <hip/hip_runtime.h>

namespace w8 {

inline void emu_land(const emu::Pending& p) {
  emu::Machine& g = emu::m();
  const unsigned at = p.lds - (unsigned)(uintptr_t)g.lds;
  if (at + p.bytes > g.lds_bytes) return emu::fault("a load past the end of LDS");
  memcpy(g.lds + at, p.data, p.bytes);
}
inline void emu_load(const void* p, unsigned lds, int bytes) {
  emu::Machine& g = emu::m();
  ++g.loads;
  emu::Pending n;
  n.lds = lds + bytes * (g.current % 64);
  n.bytes = bytes;
  memset(n.data, 0x7F, sizeof n.data);
  if (emu::inside(p, bytes))
    memcpy(n.data, p, bytes);
  else
    emu::fault("load", p, bytes);
  if (!g.opt.late) emu_land(n);
  g.fibers[g.current].loads.push_back(n);
}
inline void load_lds16(const uint8_t* p, unsigned lds) { emu_load(p, lds, 16); }
inline void load_lds16(const uint8_t* base, unsigned off, unsigned lds) {
  emu_load(base + off, lds, 16);
}
inline void load_lds4(const float* p, unsigned lds) { emu_load(p, lds, 4); }

template <int N>
inline void wait_stage() {
  emu::Machine& g = emu::m();
  std::deque<emu::Pending>& q = g.fibers[g.current].loads;
  while (q.size() > (size_t)N) {
    if (g.opt.late) emu_land(q.front());
    q.pop_front();
  }
  emu::barrier();
}

}  // namespace w8
