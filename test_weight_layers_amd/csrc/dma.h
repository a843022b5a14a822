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

// The same through a raw buffer view (wave-uniform base and byte range): BYTES (16 or 4) a lane from its own byte offset,
// zeros past the range.  The view's registers may come from VALU instructions (readfirstlane, or a spill's readlane), which a
// memory instruction may read only five wait states later: the compiler, which inserts these elsewhere, does not look into
// the asm, so they stand in it.
typedef uint32_t BufferView __attribute__((ext_vector_type(4)));
__device__ __forceinline__ BufferView untracked_view(const void *base, unsigned bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  return BufferView{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
                    (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32)) & 0xffffu,
                    (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}
template <int BYTES>
__device__ __forceinline__ void copy_to_lds_untracked(BufferView view, unsigned voffset, unsigned char *lds_wave_base) {
  static_assert(BYTES == 16 || BYTES == 4, "");
  const unsigned m0v = (unsigned)(uintptr_t)(__attribute__((address_space(3))) unsigned char *)lds_wave_base;
  if constexpr (BYTES == 16)
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(voffset), "s"(view), "{m0}"(m0v) : "memory");
  else
    asm volatile("s_nop 4\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(voffset), "s"(view), "{m0}"(m0v) : "memory");
}

}  // namespace ttt
