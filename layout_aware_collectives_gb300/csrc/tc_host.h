// Host side of the tensor-core kernels: tensor maps, and what a launch takes
// from its handle.
#pragma once

#include <cuda.h>
#include <cuda_runtime_api.h>
#include <stdint.h>

#include "compute_internal.h"

namespace tide {

// Tensor map of a row-major matrix of `elem`-byte elements, rows `ld`
// elements apart (ld * elem a multiple of 16, the pointer 16-byte aligned),
// read or written in boxes of box_cols x box_rows; outside it reads give 0
// and writes are dropped.  False if the driver refuses it.
bool make_map(CUtensorMap* map, const void* p, int elem, int64_t cols, int64_t rows, int64_t ld, uint32_t box_cols,
              uint32_t box_rows, CUtensorMapSwizzle swizzle);

// Map of a row-major bf16 matrix, `cols` a multiple of 64, as slabs of 64
// columns: coordinates (column of the slab, row, slab), boxes of two slabs by
// box_rows rows, 128-byte swizzle.
bool make_slab_map(CUtensorMap* map, const void* p, int64_t cols, int64_t rows, int64_t ld, uint32_t box_rows);

}  // namespace tide
