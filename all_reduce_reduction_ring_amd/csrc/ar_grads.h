// ar_grads.h -- launcher of the gradients' norm and clipping, and the plan that the host layer makes for it.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ar.h"

namespace ar {

struct GradArgs {
  const ar_grad_piece* pieces;
  int64_t npieces;
  double* partial;  // one per workgroup
  float* norm;
  float max_norm;
  float eps;
  int groups;
};
// clip: the elements are scaled too.
hipError_t launch_grad_norm(GradArgs a, bool max_kind, bool clip, hipStream_t s);

// Workgroups of either kernel, a function of the table alone (the order of the sum follows from it): four to a compute
// unit of 256.
constexpr int64_t kMostGroups = 1024;
constexpr int grad_groups(int64_t npieces) { return static_cast<int>(npieces < kMostGroups ? npieces : kMostGroups); }

// Bytes of a piece: two for every workgroup at least as long as that leaves them 4 KiB (a vector for each thread), and
// 32 KiB at most.
constexpr int64_t kLeastPiece = 4096, kMostPiece = 32768;
constexpr int64_t piece_bytes(int64_t total) {
  int64_t b = kLeastPiece;
  while (b < kMostPiece && total / b > 2 * kMostGroups) b *= 2;
  return b;
}

}  // namespace ar
