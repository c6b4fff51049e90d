// tensor_map.cuh -- tiled tensor maps of 16-bit strided tensors, for the serving operators.
#pragma once
#include <cuda.h>
#include <cstdint>

namespace sage {

// dims and box innermost first, strides in bytes of dims 1 .. rank-1 (multiples of 16, below 2^40);
// 128-byte swizzle, elements outside the tensor read as zero.  False when the driver's encoder is
// missing or refuses.
bool encode_tiled_16bit(CUtensorMap* map, bool bf16, const void* base, int rank, const uint64_t* dims,
                        const uint64_t* strides, const uint32_t* box);

}  // namespace sage
