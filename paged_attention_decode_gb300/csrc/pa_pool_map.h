// pa_pool_map.h -- tensor maps over the K/V pools (defined in pa_partial.cu).
#pragma once

#include <cuda.h>

#include <cstdint>

namespace pa {

// Tensor map over a pool viewed as [rows = num_pages * page_size, Hkv, D] (innermost first: D, Hkv, rows);
// a box is one KV head x `box_rows` rows x `box_d` elements of the head dim.
bool make_pool_map(CUtensorMap* map, const void* base, int dtype, int64_t rows, int hkv, int D, int box_d,
                   int box_rows, CUtensorMapSwizzle swizzle);

}  // namespace pa
