// The places that fa_page_bounds gives to the pages of a ragged batch, on the host: every page that
// holds a new key has one, no two share one, all lie in the launch, and the search finds each
// place's sequence.  Prints one line per failed check.
#include <cstdio>
#include <vector>

#include "fa_cache.h"

static int failures = 0;
#define CHECK(c) do { if (!(c)) { ++failures; std::printf("line %d: %s\n", __LINE__, #c); } } while (0)

// The search of page_bounds_kernel, lane by lane.
static int sequence_of(const int32_t* cu, int B, int total, int shift, int slot) {
  fa::OffsetSearch s{0, B};
  while (true) {
    const int step = s.step(32);
    int hits = 0;
    for (int lane = 0; lane < 32; ++lane)
      hits += lane * step < s.n && fa::first_slot(cu, s.lo + lane * step, total, shift) <= slot;
    if (hits == 0) return -1;
    s.narrow(step, hits);
    if (step == 1) return s.lo;
  }
}

int main() {
  unsigned x = 1u;
  auto random = [&](int n) {
    x = x * 1664525u + 1013904223u;
    return static_cast<int>((x >> 8) % static_cast<unsigned>(n));
  };
  for (int round = 0; round < 400; ++round)
    for (int shift = 4; shift <= 7; ++shift) {
      const int B = 1 + random(round % 7 == 0 ? 300 : 9), P = 1 << shift;
      std::vector<int32_t> cu(1, 0);
      for (int b = 0; b < B; ++b) cu.push_back(cu.back() + (random(3) == 0 ? random(2) : random(5 * P)));
      const bool single = round % 5 == 0;  // one token each
      const int32_t* offsets = single ? nullptr : cu.data();
      const int total = single ? B : cu.back();
      const int slots = (total >> shift) + 2 * B;
      std::vector<int> used(static_cast<size_t>(slots), 0);
      for (int b = 0; b < B; ++b) {
        int start, n;
        fa::token_bounds(offsets, b, total, start, n);
        const int len = random(2) ? n + random(4 * P) : random(4 * P);  // fewer keys than tokens, too
        if (n == 0 || len == 0) continue;
        const int first = (len > n ? len - n : 0) >> shift, last = (len - 1) >> shift;
        CHECK(last - first < (n >> shift) + 2);
        for (int i = 0; i <= last - first; ++i) {
          const int slot = fa::first_slot(offsets, b, total, shift) + i;
          CHECK(slot >= 0 && slot < slots);
          if (slot < 0 || slot >= slots) continue;
          CHECK(used[static_cast<size_t>(slot)]++ == 0);
          CHECK(sequence_of(offsets, B, total, shift, slot) == b);
        }
      }
    }
  std::printf(failures == 0 ? "ok\n" : "%d failures\n", failures);
  return failures == 0 ? 0 : 1;
}
