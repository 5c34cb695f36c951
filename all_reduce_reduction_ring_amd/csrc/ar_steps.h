// ar_steps.h -- sizes and byte offsets of the row copies and the steps over a token's choices: plain functions and types
// that the host layer, the kernels and the CPU tests share. A row has less than 2^31 bytes; the loops over it step past
// its end by up to a step, which 32 bits hold without a sign only.
#pragma once

#include <cstdint>

namespace ar {

using row_bytes_t = uint32_t;
constexpr row_bytes_t kVectorBytes = 16;

constexpr int64_t row_vectors(int64_t row_bytes) { return (row_bytes + kVectorBytes - 1) / kVectorBytes; }

// Bytes of the scales of a row of 8-bit codes, one float per `block` of them.
constexpr row_bytes_t row_scale_bytes(row_bytes_t hidden, row_bytes_t block) { return (hidden + block - 1) / block * 4; }

// Where the vector that starts at byte b of a row is read and written: moved up to end with the row if it runs past it.
constexpr row_bytes_t vector_place(row_bytes_t b, row_bytes_t row_bytes) {
  return b + kVectorBytes <= row_bytes ? b : row_bytes - kVectorBytes;
}

// Choices of a token handled together. A token has up to 2^31 - 1; the loops count down those that are left, which ends at
// -7 and no sum wraps. (Counted up without a sign, the combine kernel went from 113 to 179 registers and from 226 to 244 us
// at 16,384 x 8 rows of 8 KiB.)
constexpr int kChoices = 8;

// Row numbers of the sorted rows are below 2^31; a segment's pads are walked 16 rows at a time, past its end by up to 15.
using sorted_row_t = uint32_t;
constexpr int kPadLanes = 16;

// The experts' products load operand tiles in chunks of 16 bytes, also where a chunk runs past a row's end or a row lies past
// the matrix; a load stops at the number of bytes that it is given, so that number has to be exact. From a tile's base on,
// the matrix at its first row (or column) and the step's first element k of a sum of `sum`:
//   along the sum (rows of a tile lie `stride` bytes apart, all of them in the matrix): up to the end of the last of `rows`
//   across it (every element of the sum is a row of `stride` bytes, the tile starts at element `first` of it): the rest
constexpr int64_t along_left(int rows, uint32_t stride, int sum, int k, int size) {
  return static_cast<int64_t>(rows - 1) * stride + static_cast<int64_t>(sum - k) * size;
}
constexpr int64_t across_left(int sum, int k, uint32_t stride, int first, int size) {
  return static_cast<int64_t>(sum - k) * stride - static_cast<int64_t>(first) * size;
}
// As a load takes it, from its two halves. Tiles stay below 2^31 bytes, so more than that need not be told apart.
constexpr uint32_t kMostLoadBytes = 0x7FFFFFF0u;
constexpr uint32_t load_bytes(uint32_t high, uint32_t low) {
  return high != 0 ? kMostLoadBytes : low < kMostLoadBytes ? low : kMostLoadBytes;
}

// Loads through registers have no limit of their own: a chunk at byte `at` from the base is read whole where it ends within the
// `left` bytes, and element by element otherwise.
constexpr bool chunk_inside(uint32_t at, uint32_t left) { return at + 16 <= left; }

// The products of few rows walk a sum of k elements in blocks of kFewUnits times 64 bytes; behind the last whole block a lane
// takes the chunk of `v` elements at element `at` where it lies within the sum, or else what the sum's end leaves of it.
constexpr int kFewUnits = 2;
constexpr int few_block(int v) { return kFewUnits * 4 * v; }
constexpr bool few_whole(int at, int k, int v) { return at + v <= k; }

}  // namespace ar
