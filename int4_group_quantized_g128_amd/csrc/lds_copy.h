// Direct-to-LDS copies and the waits that order them (gfx950): shared by the GEMM
// kernels that stage tiles through LDS.
#pragma once
#include "common.h"

namespace q4 {

// s_waitcnt that waits until at most n vector-memory operations are outstanding
// (gfx9 encoding: vmcnt[3:0] | expcnt[6:4] | lgkmcnt[11:8] | vmcnt[5:4] in [15:14]).
template <int N>
Q4_DEVICE void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// Raw buffer resource (V#) over [base, base + bytes), bytes < 2^31: copies address it with
// a per-lane 32-bit offset plus a wave-uniform scalar offset, so advancing K costs no VALU.
Q4_DEVICE u32x4_t buffer_rsrc(const void* base, int64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4_t{uint32_t(a), uint32_t(a >> 32) & 0xffffu, uint32_t(bytes), 0x00020000u};
}

// LDS byte address of a generic pointer into LDS: the low half of a flat LDS address is
// the LDS offset (the high half is the shared aperture), so no address-space cast (and
// its null check) is needed.
Q4_DEVICE uint32_t lds_addr(const void* p) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)); }

// Direct-to-LDS copy of SIZE (16 or 4) bytes per lane: lane L's bytes land at
// lds + L * SIZE.  Written as inline asm with no register outputs other than a scratch
// SGPR: the compiler then does not see an LDS write whose target it cannot tell apart
// from the ring slot being read, and would otherwise wait for every copy in flight
// before each LDS read.  The kernel orders copies and reads itself (vmcnt waits +
// barriers).  M0 (the LDS base of the copy) is saved and restored around it; the
// leading s_nop covers the wait states between SGPR/M0 writes and their use.
template <int SIZE>
Q4_DEVICE void copy_to_lds(const u32x4_t& rsrc, uint32_t lds_in, uint32_t voff, uint32_t soff_in) {
  static_assert(SIZE == 16 || SIZE == 4, "copy size");
  // wave-uniform by construction; readfirstlane makes that visible (scalar operands)
  const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_in);
  const uint32_t soff = __builtin_amdgcn_readfirstlane(soff_in);
  uint32_t saved;
  if constexpr (SIZE == 16)
    asm volatile(
        "s_mov_b32 %0, m0\n\ts_nop 4\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
        "buffer_load_dwordx4 %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
        : "memory");
  else
    asm volatile(
        "s_mov_b32 %0, m0\n\ts_nop 4\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
        "buffer_load_dword %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
        : "memory");
  (void)saved;
}

// Two direct-to-LDS copies of 16 bytes per lane, to lds and lds + 1024 (see copy_to_lds).
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
