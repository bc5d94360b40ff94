// Loads from memory straight to LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lores {
namespace {

// 16 bytes per lane from memory (`src`, the same in all lanes, plus the lane's
// offset in bytes) straight to LDS, lane i's to `lds` + 16 i (`lds` the same in
// all lanes).  The compiler does not count these loads: arrived() waits for
// all of the wavefront's, and a barrier behind it makes them the
// work-group's.  (Written as the instruction because the builtin's wait
// before every LDS read that might alias would undo the prefetch; there is
// no output register to be overwritten in flight.)
__device__ __forceinline__ void direct16(const void *src, uint32_t lane_at, void *lds) {
    // the low half of a generic LDS address is its offset; nothing else in these
    // kernels uses m0
    const uint32_t at = (uint32_t)(uintptr_t)lds;
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :: "v"(lane_at), "s"(src), "s"(at) : "memory");
}
__device__ __forceinline__ void arrived() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

}  // namespace
}  // namespace lores
