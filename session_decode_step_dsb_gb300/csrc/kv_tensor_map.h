// Tensor maps of K and V caches and page pools viewed as [rows][D] 16-bit elements, with
// boxes of 64 columns x box_keys keys and the 128-byte swizzle; encoded on the host (no
// device work).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

namespace dsbk {

cudaError_t kv_tensor_map(const void* base, long long rows, int D, int dtype, int box_keys, CUtensorMap* out);

}  // namespace dsbk
