// Walks the loads of the experts' products' operand tiles (csrc/ar_steps.h): every chunk of 16 bytes that a tile of R rows
// loads in every step of its sum, word by word as the load's bound lets them through. No word may lie outside the matrix, and
// every element of the tile that the sum takes must come through. Arguments: element size, rows and width of the matrix.
#include <cinttypes>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "ar_steps.h"

static uint32_t allowed(int64_t left) { return ar::load_bytes(static_cast<uint32_t>(left >> 32), static_cast<uint32_t>(left)); }

static int fail(const char* what, int64_t a, int64_t b) { return printf("%s at %" PRId64 " of %" PRId64 "\n", what, a, b), 1; }

// Rows of `width` elements, the sum along them: tiles of R rows.
static int along(int size, int rows, int width, int R) {
  const int v = 16 / size, per = 8 * v;
  const uint32_t stride = static_cast<uint32_t>(width) * size;
  const int64_t all = static_cast<int64_t>(rows) * stride;
  for (int row0 = 0; row0 < rows; row0 += R) {
    const int high = rows - row0 < R ? rows - row0 : R;
    std::vector<char> seen(static_cast<size_t>(high) * stride, 0);
    for (int k = 0; k < width; k += per) {
      const int64_t base = static_cast<int64_t>(row0) * stride + static_cast<int64_t>(k) * size;
      const uint32_t bytes = allowed(ar::along_left(high, stride, width, k, size));
      for (int r = 0; r < R; ++r)
        for (int c = 0; c < 8; ++c) {
          if (k + c * v >= width) continue;
          const uint32_t at = static_cast<uint32_t>(r < high ? r : high - 1) * stride + c * 16;
          for (uint32_t w = at; w < at + 16; w += 4) {
            if (w + 4 > bytes) continue;
            if (base + w + 4 > all) return fail("a load past the matrix", base + w, all);
            const int64_t in_tile = base + w - static_cast<int64_t>(row0) * stride;
            if (r < high && in_tile < static_cast<int64_t>(r + 1) * stride)
              for (int i = 0; i < 4; ++i) seen[in_tile + i] = 1;
          }
        }
    }
    for (size_t i = 0; i < seen.size(); ++i)
      if (!seen[i]) return fail("an element that no load brings", i, seen.size());
  }
  return 0;
}

// The sum over the rows (`sum` of them; more lie behind), tiles of R elements of a row.
static int across(int size, int sum, int width, int R) {
  const int v = 16 / size, per = 8 * v;
  const uint32_t stride = static_cast<uint32_t>(width) * size;
  const int64_t all = static_cast<int64_t>(sum) * stride;
  for (int first = 0; first < width; first += R) {
    std::vector<char> seen(static_cast<size_t>(all), 0);
    for (int k = 0; k < sum; k += per) {
      const int64_t base = static_cast<int64_t>(k) * stride + static_cast<int64_t>(first) * size;
      const uint32_t bytes = allowed(ar::across_left(sum, k, stride, first, size));
      for (int r = 0; r < per; ++r)
        for (int c = 0; c < R / v; ++c) {
          const uint32_t at = static_cast<uint32_t>(r) * stride + c * 16;
          for (uint32_t w = at; w < at + 16; w += 4) {
            if (w + 4 > bytes) continue;
            if (base + w + 4 > all) return fail("a load past the matrix", base + w, all);
            if (k + r >= sum) return fail("a row past the sum", k + r, sum);
            const int64_t end = static_cast<int64_t>(k + r + 1) * stride;
            for (int i = 0; i < 4; ++i)
              if (base + w + i < end) seen[base + w + i] = 1;
          }
        }
    }
    for (int k = 0; k < sum; ++k)
      for (int64_t b = static_cast<int64_t>(first) * size; b < stride && b < static_cast<int64_t>(first + R) * size; ++b)
        if (!seen[static_cast<int64_t>(k) * stride + b]) return fail("an element that no load brings", k, b);
  }
  return 0;
}

int main(int argc, char** argv) {
  const int size = atoi(argv[1]), rows = atoi(argv[2]), width = atoi(argv[3]);
  int bad = 0;
  for (int R : {64, 128, 256}) bad |= along(size, rows, width, R) | across(size, rows, width, R);
  // bounds past 32 bits
  const int64_t far = ar::along_left(256, 4u << 20, 1 << 20, 0, 4);
  bad |= allowed(far) != far || allowed(int64_t(1) << 33) != ar::kMostLoadBytes ||
         allowed(ar::across_left(2147483647, 0, 4u << 20, 0, 4)) != ar::kMostLoadBytes;
  return argc != 4 || bad;
}
