// Direct-to-LDS loads and the waits that go with them, in gfx950 assembly.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w8 {

// (the compiler says of M0 below that it keeps no value there across such a
// statement, which is what naming it is for)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"

// Direct-to-LDS loads: lane i's 16 (or 4) bytes go to LDS byte lds + 16 i (or
// 4 i).  M0 carries the LDS address and needs one wait state before its use.
// Written as assembly because the compiler, which cannot tell the stages of
// the LDS buffer apart, would wait for every load in flight before each LDS
// read; wait_stage() below does the waiting, and as volatile assembly the two
// keep their order.
// The address is a 64-bit one per lane, or a uniform base and a 32-bit offset
// per lane.  The base is copied by a scalar move on the way: a load may not
// read a scalar register within five wait states of a vector instruction's
// write to it, which the compiler does not watch in assembly (and the move is
// M0's wait state too).
__device__ __forceinline__ void load_lds16(const uint8_t* p, unsigned lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(lds), "v"(p)
               : "m0");
}
__device__ __forceinline__ void load_lds16(const uint8_t* base, unsigned off, unsigned lds) {
  const uint8_t* copy;
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\tglobal_load_lds_dwordx4 %2, %0"
               : "=&s"(copy)
               : "s"(lds), "v"(off), "s"(base)
               : "m0");
}
__device__ __forceinline__ void load_lds4(const float* p, unsigned lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(lds), "v"(p)
               : "m0");
}
#pragma clang diagnostic pop

// Waits until at most N of this wave's loads are in flight and its LDS reads
// have returned, then for the workgroup's other waves.
template <int N>
__device__ __forceinline__ void wait_stage() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

}  // namespace w8
