// Reads through a request's block table, shared by the paged kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rts_internal.h"

namespace rts {

// Physical row of position `pos` (>= 0) of the request whose block-table row
// is `row`; -1 where there is none: a block past the table, a negative block
// id, or a physical row outside the cache.
__device__ __forceinline__ int64_t phys_row(const Pages& pg, const int32_t* row, int32_t pos) {
    const uint32_t p = (uint32_t)pos;
    const uint32_t b = pg.shift >= 0 ? p >> pg.shift : p / (uint32_t)pg.block_size;
    if (b >= (uint32_t)pg.cols) return -1;
    const int32_t id = row[b];
    if (id < 0) return -1;
    const int64_t r = (int64_t)id * pg.stride_rows + (p - b * (uint32_t)pg.block_size);
    return r < pg.cache_rows ? r : -1;
}

}  // namespace rts
