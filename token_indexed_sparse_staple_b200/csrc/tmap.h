// Tensor maps for the TMA copies, shared by the launchers (not part of the
// public ABI).
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace stp {

// Map of a row-major matrix of `rows` rows of `cols` elements (row pitch ld
// elements, esize bytes each), box = box_cols x box_rows; what a copy reads
// outside the matrix is zero.  False if the driver refuses it.
bool tensor_map_2d(CUtensorMap* m, CUtensorMapDataType type, int esize, const void* base,
                   uint64_t cols, uint64_t rows, uint64_t ld, uint32_t box_cols, uint32_t box_rows,
                   CUtensorMapSwizzle swizzle);

}  // namespace stp
