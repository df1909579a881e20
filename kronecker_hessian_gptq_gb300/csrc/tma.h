// tma.h -- host side of the tiled TMA copies: tensor maps of row-major matrices.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace bakron {

// A row-major rows x cols matrix of 8- or 16-bit elements with a row stride
// of ld elements, copied in boxes of box_rows x box_cols into shared memory,
// swizzled by 128 bytes (a box row is then 128 bytes) or not.
// The base and the stride have to be multiples of 16 bytes; what a box covers
// outside the matrix reads as zeros.
struct TileMap {
  const void* base;
  CUtensorMapDataType type;
  int64_t rows, cols, ld;
  uint32_t box_rows, box_cols;
  bool swizzle;
};
cudaError_t make_tensor_map(CUtensorMap* out, const TileMap& t);

}  // namespace bakron
