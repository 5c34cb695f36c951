// Walks the last 100 rows of a segment that ends at the row given, 16 lanes at a time (csrc/ar_steps.h) as the sort does:
// every row once, none outside, and every lane's walk ends.
#include <cinttypes>
#include <cstdio>
#include <cstdlib>

#include "ar_steps.h"

int main(int argc, char** argv) {
  for (int i = 1; i < argc; ++i) {
    const int64_t last = strtoll(argv[i], nullptr, 10), first = last > 100 ? last - 100 : 0;
    int64_t rows = 0;
    for (int lane = 0; lane < ar::kPadLanes; ++lane) {
      const ar::sorted_row_t end = static_cast<ar::sorted_row_t>(last);
      for (ar::sorted_row_t p = static_cast<ar::sorted_row_t>(first) + lane; p < end; p += ar::kPadLanes) {
        const int64_t at = p;
        if (at < first || at >= last || ++rows > last - first) return printf("%" PRId64 ": row %" PRId64 "\n", last, at), 1;
      }
    }
    if (rows != last - first) return printf("%" PRId64 ": %" PRId64 " rows\n", last, rows), 1;
  }
  return 0;
}
