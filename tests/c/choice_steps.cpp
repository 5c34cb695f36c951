// Steps over the choices of a token (csrc/ar_steps.h) as the kernels do, for counts given as arguments: the walk takes
// every choice once and ends.
#include <cinttypes>
#include <cstdio>
#include <cstdlib>

#include "ar_steps.h"

int main(int argc, char** argv) {
  for (int i = 1; i < argc; ++i) {
    const int64_t count = strtoll(argv[i], nullptr, 10);
    const ar::choice_t k = static_cast<ar::choice_t>(count);
    int64_t n = 0;
    for (ar::choice_t j0 = 0; j0 < k; j0 += ar::kChoices) {
      if (static_cast<int64_t>(j0) != n * ar::kChoices || ++n > (count + ar::kChoices - 1) / ar::kChoices)
        return printf("%" PRId64 ": step %" PRId64 " at %" PRId64 "\n", count, n, static_cast<int64_t>(j0)), 1;
    }
    if (n != (count + ar::kChoices - 1) / ar::kChoices) return printf("%" PRId64 ": %" PRId64 " steps\n", count, n), 1;
  }
  return 0;
}
