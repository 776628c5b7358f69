// Reads through a request's block table and loads straight into LDS, shared by
// the kernels that stream a cache.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rts_internal.h"

namespace rts {

// The block of position e.
__device__ __forceinline__ uint32_t block_of(const Pages& pg, uint32_t e) {
    return pg.shift >= 0 ? e >> pg.shift : e / (uint32_t)pg.block_size;
}

// Physical row of position e, whose block-table entry is `entry`; -1 where
// there is none: a block past the table, a negative block id, or a physical
// row outside the cache (of fewer than 2^31 rows).
__device__ __forceinline__ int phys_row(const Pages& pg, int entry, uint32_t e) {
    const uint32_t b = block_of(pg, e);
    const int64_t r = (int64_t)entry * pg.stride_rows + (e - b * (uint32_t)pg.block_size);
    return entry >= 0 && b < (uint32_t)pg.cols && r < pg.cache_rows ? (int)r : -1;
}

// LDS by its byte address.
template <typename T>
__device__ __forceinline__ T lds_read(uint32_t at) {
    return *(const __attribute__((address_space(3))) T*)(uintptr_t)at;
}
__device__ __forceinline__ uint32_t lds_address(const char* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// SIZE bytes a lane from global memory, src + OFFSET, to LDS at base + OFFSET +
// SIZE * lane.  Written in assembly (no register is loaded) because the
// compiler cannot tell the stages of a ring apart: with the builtin it waits
// for every load under way before it reads any stage.  The callers count the
// loads and wait themselves; all of them have arrived before a workgroup ends.
template <int SIZE, int OFFSET>
__device__ __forceinline__ void load_to_lds(const char* src, uint32_t base) {
    if constexpr (SIZE == 16)
        asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off offset:%2" ::"{m0}"(base), "v"(src), "n"(OFFSET)
                     : "memory");
    else
        asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, off offset:%2" ::"{m0}"(base), "v"(src), "n"(OFFSET)
                     : "memory");
}

}  // namespace rts
