// Walks the loads of the experts' products that go through registers (csrc/ar_steps.h): operand tiles of rows of any width, and
// the kernel for few rows. Element by element as the kernels read them: none may lie outside the matrix, and every element of
// the sum must come through, once. Arguments: element size, rows and width of the matrix.
#include <cinttypes>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "ar_steps.h"

static uint32_t limit_of(int64_t left) { return ar::load_bytes(static_cast<uint32_t>(left >> 32), static_cast<uint32_t>(left)); }

static int fail(const char* what, int64_t a, int64_t b) { return printf("%s at %" PRId64 " of %" PRId64 "\n", what, a, b), 1; }

// `n` elements from byte `at` of a matrix of `all` bytes.
static bool outside(int64_t at, int n, int size, int64_t all) { return n > 0 && (at < 0 || at + static_cast<int64_t>(n) * size > all); }

// Rows of `width` elements, the sum along them: tiles of R rows, chunks that the row's end cuts masked behind it.
static int along(int size, int rows, int width, int R) {
  const int v = 16 / size, per = 8 * v;
  const uint32_t stride = static_cast<uint32_t>(width) * size;
  const int64_t all = static_cast<int64_t>(rows) * stride;
  for (int row0 = 0; row0 < rows; row0 += R) {
    const int high = rows - row0 < R ? rows - row0 : R;
    std::vector<char> seen(static_cast<size_t>(high) * width, 0);
    for (int k = 0; k < width; k += per) {
      const int64_t base = static_cast<int64_t>(row0) * stride + static_cast<int64_t>(k) * size;
      const uint32_t left = limit_of(ar::along_left(high, stride, width, k, size));
      for (int r = 0; r < R; ++r)
        for (int c = 0; c < 8; ++c) {
          const int n = width - k - c * v;
          if (n <= 0) continue;
          const uint32_t at = static_cast<uint32_t>(r < high ? r : high - 1) * stride + c * 16;
          const int take = ar::chunk_inside(at, left) ? v : n < v ? n : v;
          if (outside(base + at, take, size, all)) return fail("a load past the matrix", base + at, all);
          for (int i = 0; r < high && i < take && i < n; ++i) ++seen[static_cast<size_t>(r) * width + k + c * v + i];
        }
    }
    for (size_t i = 0; i < seen.size(); ++i)
      if (seen[i] != 1) return fail("an element that does not come through once", i, seen.size());
  }
  return 0;
}

// The sum over the rows, tiles of R elements of a row.
static int across(int size, int sum, int width, int R) {
  const int v = 16 / size, per = 8 * v;
  const uint32_t stride = static_cast<uint32_t>(width) * size;
  const int64_t all = static_cast<int64_t>(sum) * stride;
  for (int first = 0; first < width; first += R) {
    std::vector<char> seen(static_cast<size_t>(sum) * width, 0);
    for (int k = 0; k < sum; k += per) {
      const int64_t base = static_cast<int64_t>(k) * stride + static_cast<int64_t>(first) * size;
      const uint32_t left = limit_of(ar::across_left(sum, k, stride, first, size));
      for (int r = 0; r < per; ++r)
        for (int c = 0; c < R; c += v) {
          if (k + r >= sum) continue;
          const uint32_t at = static_cast<uint32_t>(r) * stride + c * size;
          const int n = width - first - c, take = ar::chunk_inside(at, left) ? v : n < 0 ? 0 : n < v ? n : v;
          if (outside(base + at, take, size, all)) return fail("a load past the matrix", base + at, all);
          for (int i = 0; i < take && i < n; ++i) ++seen[static_cast<size_t>(k + r) * width + first + c + i];
        }
    }
    for (int k = 0; k < sum; ++k)
      for (int c = first; c < width && c < first + R; ++c)
        if (seen[static_cast<size_t>(k) * width + c] != 1) return fail("an element that does not come through once", k, c);
  }
  return 0;
}

// Few rows: four waves in turn over the blocks from block `turn` on, the next block ahead of this one's products.
static int few(int size, int rows, int width, int tile, int turn) {
  const int v = 16 / size, block = ar::few_block(v), blocks = width / block, waves = 4;
  const int64_t stride = static_cast<int64_t>(width) * size, all = rows * stride;
  if (blocks > 0) turn %= blocks;
  for (int row0 = 0; row0 < rows; row0 += tile) {
    std::vector<char> seen(static_cast<size_t>(tile) * width, 0);
    int bad = 0;
    for (int wave = 0; wave < waves; ++wave) {
      auto load = [&](int b) {
        b += turn;
        const int from = (b >= blocks ? b - blocks : b) * block;
        for (int r = 0; r < tile; ++r)
          for (int u = 0; u < ar::kFewUnits; ++u)
            for (int q = 0; q < 4; ++q) {
              const int row = row0 + r < rows ? row0 + r : rows - 1, e = from + u * 4 * v + q * v;
              bad |= outside(row * stride + static_cast<int64_t>(e) * size, v, size, all) || e + v > width;
              for (int i = 0; !bad && i < v; ++i) ++seen[static_cast<size_t>(r) * width + e + i];
            }
      };
      int b = wave;
      if (b < blocks) load(b);
      for (; b < blocks; b += 2 * waves) {
        if (b + waves < blocks) load(b + waves);
        if (b + 2 * waves < blocks) load(b + 2 * waves);
      }
      const int rest = blocks * block + wave * 4 * v;
      for (int q = 0; rest < width && q < 4; ++q) {
        const int k = rest + q * v, n = ar::few_whole(k, width, v) ? v : k < width ? width - k : 0;
        for (int r = 0; r < tile; ++r) {
          const int row = row0 + r < rows ? row0 + r : rows - 1;
          bad |= n > 0 && (outside(row * stride + static_cast<int64_t>(k) * size, n, size, all) || k + n > width);
          for (int i = 0; !bad && i < n && i < v; ++i) ++seen[static_cast<size_t>(r) * width + k + i];
        }
      }
      if (bad) return fail("a load past the matrix or the row", row0, wave);
    }
    for (size_t i = 0; i < seen.size(); ++i)
      if (seen[i] != 1) return fail("an element that does not come through once", i, seen.size());
  }
  return 0;
}

int main(int argc, char** argv) {
  const int size = atoi(argv[1]), rows = atoi(argv[2]), width = atoi(argv[3]);
  int bad = 0;
  for (int R : {64, 128}) bad |= along(size, rows, width, R) | across(size, rows, width, R);
  for (int tile : {16, 32})
    for (int turn : {0, 1, 9, 100}) bad |= few(size, rows, width, tile, turn);
  return argc != 4 || bad;
}
