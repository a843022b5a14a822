// Copies from memory to LDS that the compiler does not count.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ttt {

// copy16_to_lds (global_load_lds_dwordx4) issued through inline asm, so that the
// compiler does not count it: its waits for LDS reads cannot tell which stage a
// pending copy writes once the copies stay in flight across a loop's back edge, and
// it then waits for all of them.  The caller waits for these copies itself
// (s_waitcnt vmcnt) before reading their data.
__device__ __forceinline__ void copy16_to_lds_untracked(const void *gsrc, unsigned char *lds_wave_base) {
  const unsigned m0v = (unsigned)(uintptr_t)(__attribute__((address_space(3))) unsigned char *)lds_wave_base;
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(gsrc), "{m0}"(m0v) : "memory");
}

}  // namespace ttt
