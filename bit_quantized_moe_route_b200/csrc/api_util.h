// Host helpers of the C ABI shared by its translation units (defined in moe_api.cu).
#pragma once

#include <cuda.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_lowbit.h"

namespace moe {

// Records the calling thread's error detail and returns `st`.
moe_status_t api_fail(moe_status_t st, const char* fmt, ...);
void api_clear_detail();
// Device (or managed) memory, not NULL.
moe_status_t api_check_dev_ptr(const void* p, const char* name);
// Tiled tensor map of rank 2 or 3: dims and box in elements (dims[0] contiguous),
// strides in bytes for dims 1.., 128-byte swizzle or none, zero fill out of bounds.
moe_status_t api_tensor_map(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* ptr, const uint64_t* dims,
                            const uint64_t* strides, const uint32_t* box, bool swizzle = true);

}  // namespace moe
