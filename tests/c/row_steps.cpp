// Walks the row copy's steps (csrc/ar_steps.h) as a workgroup of 128 lanes with four 16-byte vectors each does, for row
// sizes given as arguments, and checks that every vector lies in the row, that the vectors of a step follow one another,
// and that the walk ends behind the row's last byte.
#include <cinttypes>
#include <cstdio>
#include <cstdlib>

#include "ar_steps.h"

static int walk(int64_t row64) {
  constexpr ar::row_bytes_t kLanes = 128, kVectors = 4;
  const ar::row_bytes_t row = static_cast<ar::row_bytes_t>(row64);
  const ar::row_bytes_t lanes[] = {0, 1, 63, 64, kLanes - 1};
  const int64_t steps = (row64 + kLanes * kVectors * 16 - 1) / (kLanes * kVectors * 16);
  for (ar::row_bytes_t lane : lanes) {
    int64_t n = 0, covered = 0;
    for (ar::row_bytes_t b0 = lane * 16; b0 < row; b0 += kLanes * kVectors * 16) {
      if (++n > steps) return printf("%" PRId64 ", lane %u: more steps than the row has\n", row64, (unsigned)lane), 1;
      for (ar::row_bytes_t u = 0; u < kVectors; ++u) {
        const int64_t want = (n - 1) * kLanes * kVectors * 16 + lane * 16 + u * kLanes * 16;
        const int64_t at = static_cast<uint32_t>(ar::vector_place(b0 + u * kLanes * 16, row));
        if (at != (want + 16 <= row64 ? want : row64 - 16)) return printf("%" PRId64 ": vector of byte %" PRId64 " at %" PRId64 "\n", row64, want, at), 1;
        if (want < row64) covered = at + 16;
      }
    }
    const int64_t last = (row64 - 1) / 16 * 16 - lane * 16;  // the row's last vector, where it is this lane's
    if (last >= 0 && last % (kLanes * 16) == 0 && covered != row64) return printf("%" PRId64 ": ends at %" PRId64 "\n", row64, covered), 1;
  }
  if (ar::row_vectors(row64) != (row64 + 15) / 16) return printf("%" PRId64 ": vectors\n", row64), 1;
  if (static_cast<int64_t>(ar::row_scale_bytes(row, 128)) != (row64 + 127) / 128 * 4) return printf("%" PRId64 ": scales\n", row64), 1;
  return 0;
}

int main(int argc, char** argv) {
  for (int i = 1; i < argc; ++i)
    if (walk(strtoll(argv[i], nullptr, 10))) return 1;
  return 0;
}
