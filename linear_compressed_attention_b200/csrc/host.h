// Host state shared by the library's translation units (not part of the C ABI).
#pragma once

#include <cuda.h>

namespace edit {

// Adds one to the calling thread's edit_attn_kernel_launches().
void count_launch();
// SM count of the current device (148 when none is visible).
int device_sms();
// Tensor map of a bf16 tensor, 128-byte swizzle, zero fill.
bool bf16_tensor_map(CUtensorMap* m, int rank, const void* base, const cuuint64_t* dims,
                     const cuuint64_t* strides_bytes, const cuuint32_t* box);

}  // namespace edit
