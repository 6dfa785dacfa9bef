// How the paged kernels' work is described, called on the host: the spans that the join reads.
// Prints one line per failed check.
#include <cstdio>

#include "fa_paged.h"

static int failures = 0;
#define CHECK(c) do { if (!(c)) { ++failures; std::printf("line %d: %s\n", __LINE__, #c); } } while (0)

// every span whose workers exist, and none besides
static void spans() {
  for (int workers : {0, 1, 2, 152, 1216})
    for (int first = -2; first < workers + 3; ++first)
      for (int count = -2; count < workers + 3; ++count) {
        bool all = count >= 1;  // each worker of the span exists
        for (int i = 0; i < count; ++i) all = all && first + i >= 0 && first + i < workers;
        CHECK(fa::span_ok(first, count, workers) == all);
      }
  // what a workspace may hold where no span was written: sums that leave 32 bits among it
  const int odd[][2] = {{1, 0x7fffffff}, {0x7fffffff, 2}, {-5, 3}, {0x7fffffff, 0x7fffffff},
                        {-0x7fffffff - 1, 1}, {0, -0x7fffffff - 1}, {1215, 0x7fffffff}};
  for (const auto& s : odd)
    for (int workers : {0, 1, 152, 1216}) CHECK(!fa::span_ok(s[0], s[1], workers));
  CHECK(fa::span_ok(1215, 1, 1216) && !fa::span_ok(1215, 2, 1216) && fa::span_ok(0, 1216, 1216));
}

int main() {
  spans();
  if (failures == 0) std::printf("ok\n");
  return failures != 0;
}
