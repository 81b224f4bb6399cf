// Tensor maps of the 8-bit cache's codes (fp8_maps.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace pkv {

// A tiled map of bytes, innermost dim first; strides of the dims behind it in bytes.
cudaError_t encode_code_map(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                            const cuuint32_t* box, CUtensorMapSwizzle swizzle);

}  // namespace pkv
