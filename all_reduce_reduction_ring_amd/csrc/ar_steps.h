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

}  // namespace ar
