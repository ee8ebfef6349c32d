// Direct-to-LDS copies for the dense products.
#pragma once
#include "common.h"

namespace q4 {

// LDS byte address of a generic pointer into LDS (the low half of a flat LDS address).
Q4_DEVICE uint32_t lds_addr(const void* p) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)); }

// Copies 16 bytes per lane from the buffer (a raw buffer descriptor; offsets past its range
// read zeros) to lds + 16 lane; copy2_to_lds also a second set to lds + 1024 + 16 lane.
// Inline asm with no register outputs but a scratch SGPR, so that the compiler does not wait
// for copies in flight before LDS reads of other slots: the kernels order copies and reads
// themselves (vmcnt waits and barriers).  M0, the LDS base of a copy, is saved and restored;
// the first s_nop covers an SGPR written just before by a vector instruction.
Q4_DEVICE void copy_to_lds(const u32x4_t& rsrc, uint32_t lds_in, uint32_t voff) {
  const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_in);   // wave-uniform by construction
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_nop 4\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
      "buffer_load_dwordx4 %2, %3, 0 offen lds\n\ts_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(lds), "v"(voff), "s"(rsrc)
      : "memory");
  (void)saved;
}
Q4_DEVICE void copy2_to_lds(const u32x4_t& rsrc, uint32_t lds_in, uint32_t voff0, uint32_t voff1) {
  const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_in);
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_nop 4\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
      "buffer_load_dwordx4 %2, %4, 0 offen lds\n\ts_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
      "buffer_load_dwordx4 %3, %4, 0 offen lds\n\ts_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(lds), "v"(voff0), "v"(voff1), "s"(rsrc)
      : "memory", "scc");
  (void)saved;
}

}  // namespace q4
