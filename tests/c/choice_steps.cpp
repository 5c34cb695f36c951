// Steps over the choices of a token (csrc/ar_steps.h) as the kernels do, counting down what is left, for counts given as
// arguments: the walk takes every choice once and ends. COUNT_UP: counting up instead.
#include <cinttypes>
#include <cstdio>
#include <cstdlib>

#include "ar_steps.h"

static bool step(int64_t count, int64_t* n, int j0) {
  return j0 == *n * ar::kChoices && ++*n <= (count + ar::kChoices - 1) / ar::kChoices;
}

int main(int argc, char** argv) {
  for (int i = 1; i < argc; ++i) {
    const int64_t count = strtoll(argv[i], nullptr, 10);
    const int k = static_cast<int>(count);
    int64_t n = 0;
#ifdef COUNT_UP
    for (int j0 = 0; j0 < k; j0 += ar::kChoices) {
#else
    for (int left = k; left > 0; left -= ar::kChoices) {
      const int j0 = k - left;
#endif
      if (!step(count, &n, j0)) return printf("%" PRId64 ": step %" PRId64 " at %d\n", count, n, j0), 1;
    }
    if (n != (count + ar::kChoices - 1) / ar::kChoices) return printf("%" PRId64 ": %" PRId64 " steps\n", count, n), 1;
  }
  return 0;
}
