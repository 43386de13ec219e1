// mxfp4_tile.h — copies from global memory straight into LDS, and the order of
// tiles over the chip, shared by the tiled MXFP4 products.  Private to libmxfp4.
#pragma once

#include "mxfp4_device.h"

namespace mxfp4 {

typedef __attribute__((address_space(3))) char lds_char;
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(lds_char*)p;
}

// Memory a buffer instruction may touch: `bytes` from p on.  Loads past the
// end return 0.
__device__ __forceinline__ uint4_t make_rsrc(const void* p, uint32_t bytes) {
    const uint64_t b = (uint64_t)p;
    return (uint4_t){(uint32_t)b, (uint32_t)(b >> 32) & 0xFFFFu, bytes, 0x00020000u};
}

// 16 bytes per lane from rsrc base + voff into LDS at lds + 16 * lane (lds and
// rsrc the same in the wave).  No register is written: the copy
// is complete once the wave's load counter has passed it (wait_copies).
// Written as assembly because the compiler waits for every such copy in flight
// before any LDS read.  The five wait states are those between a lane-read
// SGPR and a memory instruction that uses it.
__device__ __forceinline__ void copy16(uint4_t rsrc, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc)
                 : "m0", "memory");
}
// The same from a 64-bit address per lane.
__device__ __forceinline__ void copy16(const void* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(lds), "v"(p)
                 : "m0", "memory");
}
// The same from a base (the same in the wave) and an offset of a lane in bytes.
__device__ __forceinline__ void copy16(const void* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(base)
                 : "m0", "memory");
}
// Four bytes per lane, into LDS at lds + 4 * lane.
__device__ __forceinline__ void copy4(const void* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(base)
                 : "m0", "memory");
}
// Waits until at most `left` of the wave's loads are in flight and its LDS
// operations are done, then for the block's other waves.
template <int LEFT>
__device__ __forceinline__ void wait_copies() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

// Which tile block `id` of `total` takes.  Blocks are dealt to the 8 XCDs in
// turn; XCD x gets a contiguous run of tiles, so that what it reads stays in
// its own L2.
__device__ __forceinline__ int xcd_order(int id, int total) {
    const int q = total / 8, r = total % 8, x = id % 8;
    return x * q + min(x, r) + id / 8;
}

}  // namespace mxfp4
