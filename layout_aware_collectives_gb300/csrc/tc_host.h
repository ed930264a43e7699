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

// Division of whole numbers below 2^31 by one that a launch knows: with m =
// floor(2^63 / d) + 1 the quotient is floor(t m / 2^63), as t (m d - 2^63) <
// 2^63.
struct Divisor {
  uint64_t m;
  int d;

  Divisor() = default;
  explicit Divisor(int by) : m((1ull << 63) / (uint64_t)by + 1), d(by) {}
#ifdef __CUDACC__
  __device__ __forceinline__ int of(int t) const { return (int)__umul64hi((uint64_t)t << 1, m); }
#endif
};

// Tiles of one or several products, in bands of 16 down the rows, so that the
// tiles at work at one time share their operands in L2.
constexpr int kBand = 16;
struct TileGrid {
  int tiles_m, tiles_n;
  Divisor all, band, last;  // tiles of a product, of a band; rows of the last band

  TileGrid() = default;
  TileGrid(int m, int n)
      : tiles_m(m), tiles_n(n), all(m * n), band(kBand * n), last(m % kBand ? m % kBand : kBand) {}
};

}  // namespace tide
