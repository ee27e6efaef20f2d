// Host helpers shared by the library's entry points (defined in dropkv_api.cu).
#pragma once
#include <cstddef>
#include <cuda.h>

namespace dropkv {

// SM count of the current device, -1 without one.
int current_sms(int* dev_out);
// Tensor map of a bf16 [depth][n_max][d] array in boxes of 64 columns x 128 rows, 128-byte swizzled.
bool encode_rows(CUtensorMap* map, const void* base, int d, int n_max, int depth);
bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb);

}  // namespace dropkv
