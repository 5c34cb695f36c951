// ar_products.h -- launchers of the experts' products, and the number of tiles that a call can have, which the host layer
// checks against what the kernels count in.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ar {

struct ProductArgs {
  // gated: a0 the rows x, b0 and b1 w_gate and w_up, c0 h, c1 and c2 g and u (or null)
  // linear: a0 x, b0 w, c0 y
  // input: a0 dy, b0 w, c0 dx; with a1 and b1 a second product in the same sum
  // weight: a0 dy, b0 x, c0 dw; a1 and c1 (or null) a second gradient against the same x
  // slopes: a0 dh, b0 g, b1 u, c0 dg, c1 du
  const void* a0;
  const void* a1;
  const void* b0;
  const void* b1;
  void* c0;
  void* c1;
  void* c2;
  const int32_t* offsets;  // null: one segment of all rows
  const int32_t* counts;   // null: a segment goes up to the next offset
  int64_t w_stride;        // elements between the experts' matrices in b0 and b1
  int64_t c_stride;        // the same in c0 and c1 of weight
  int rows;                // of the sorted buffers
  int experts;
  int m;                   // weight: rows of a matrix
  int n;                   // columns of the result
  int k;                   // elements of a sum (weight: the segment's rows instead)
  int act;
  int most;                // set by the launchers: no tables give more tiles of rows
};

hipError_t launch_gated(const ProductArgs& a, int dtype, hipStream_t s);
hipError_t launch_linear(const ProductArgs& a, int dtype, hipStream_t s);
hipError_t launch_input_grad(const ProductArgs& a, int dtype, hipStream_t s);
hipError_t launch_weight_grad(const ProductArgs& a, int dtype, hipStream_t s);
hipError_t launch_slopes(ProductArgs a, int dtype, hipStream_t s);

constexpr int64_t tiles_up(int64_t v, int64_t unit) { return (v + unit - 1) / unit; }
// The most tiles of `unit` elements that the segments of rows of `width` elements have: one of each expert with rows may
// not be full.
inline int64_t row_tiles(const ProductArgs& a, int64_t width, int64_t unit) {
  if (!a.offsets) return tiles_up(a.rows * width, unit);
  return a.rows * width / unit + (a.experts < a.rows ? a.experts : a.rows);
}
inline int64_t matrices(const ProductArgs& a) { return static_cast<int64_t>(a.experts) * (a.a1 ? 2 : 1); }

// Kernels count tiles in 32 bits and step past the last one by a grid. The smallest tiles are 16 columns wide or high.
constexpr int64_t kMostTiles = int64_t(1) << 30;

}  // namespace ar
