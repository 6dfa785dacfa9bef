// The index functions that the paged kernels share, called on the host: bad pages, tokens of
// ragged batches, and the row tiles of the partial results.  Prints one line per failed check.
#include <cstdio>
#include <vector>

#include "fa_paged.h"
#include "paged_plan.cuh"

static int failures = 0;
#define CHECK(c) do { if (!(c)) { ++failures; std::printf("line %d: %s\n", __LINE__, #c); } } while (0)

int main() {
  // pages: entries below zero, past the pool, past the table; negative keys
  const int32_t row[4] = {7, -1, 8, 0};
  for (int shift = 4; shift <= 7; ++shift) {
    const int p = 1 << shift;
    CHECK(fa::resolve_page(row, 4, 8, shift, 0) == 7);
    CHECK(fa::resolve_page(row, 4, 8, shift, p - 1) == 7);
    CHECK(fa::resolve_page(row, 4, 8, shift, p) == -1);          // entry -1
    CHECK(fa::resolve_page(row, 4, 8, shift, 2 * p) == -1);      // 8 of 8 pages
    CHECK(fa::resolve_page(row, 4, 9, shift, 2 * p) == 8);
    CHECK(fa::resolve_page(row, 4, 8, shift, 4 * p - 1) == 0);
    CHECK(fa::resolve_page(row, 4, 8, shift, 4 * p) == -1);      // past the table
    CHECK(fa::resolve_page(row, 4, 8, shift, 0x7fffffff) == -1);
    CHECK(fa::resolve_page(row, 4, 8, shift, -1) == -1);
    CHECK(fa::resolve_page(nullptr, 0, 8, shift, 0) == -1);      // empty table
  }
  // tokens of a ragged batch with empty sequences and tokens behind the last one
  const int32_t cu[6] = {0, 0, 3, 3, 4, 4};
  for (int t = -1; t < 8; ++t) {
    int want = -1;
    for (int b = 0; b < 5; ++b)
      if (t >= cu[b] && t < cu[b + 1]) want = b;
    CHECK(fa::token_sequence(cu, 5, t) == want);
  }
  CHECK(fa::token_sequence(nullptr, 3, 2) == 2 && fa::token_sequence(nullptr, 3, 3) == -1);
  // offsets that are not what they should be stay inside the tensor
  const int32_t bad[5] = {-4, 9, 2, 100, 5};
  for (int b = 0; b < 4; ++b) {
    int start, n;
    fa::token_bounds(bad, b, 10, start, n);
    CHECK(start >= 0 && n >= 0 && start + n <= 10);
  }
  // row tiles of consecutive entries never overlap and stay inside the bound
  for (int R : {16, 128, 256})
    for (int G : {1, 3, 4, 5, 8, 32, 128})
      for (int seed = 0; seed < 50; ++seed) {
        std::vector<int32_t> c(1, 0);
        unsigned x = 12345u + 97u * seed;
        const int B = 1 + seed % 9;
        for (int b = 0; b < B; ++b) {
          x = x * 1664525u + 1013904223u;
          c.push_back(c.back() + static_cast<int>((x >> 16) % (seed % 3 == 0 ? 3 : 60)));
        }
        const int total = c.back(), bound = fa::row_tiles_bound(total, G, R, B);
        int used = 0;
        for (int b = 0; b < B; ++b) {
          int start, n;
          fa::token_bounds(c.data(), b, total, start, n);
          const int t0 = fa::row_tile0(start, G, R, b), rt = (n * G + R - 1) / R;
          if (rt == 0) continue;
          CHECK(t0 >= used);
          used = t0 + rt;
          CHECK(used <= bound);
        }
      }
  // shares of C CTAs: contiguous, as equal as can be, and the owner of a unit is the CTA whose
  // share holds it
  const int sizes[][2] = {{7, 1}, {16, 16}, {16, 152}, {152, 152}, {153, 152}, {303, 152},
                          {65536, 152}, {12345, 77}, {0x7fffffff, 152}, {0x7fffffff, 1}};
  for (const auto& wc : sizes) {
    const int W = wc[0], C = wc[1] < W ? wc[1] : W;
    CHECK(fa::share_begin(W, C, 0) == 0 && fa::share_begin(W, C, C) == W);
    for (int k = 0; k < C; ++k) {
      const int u0 = fa::share_begin(W, C, k), u1 = fa::share_begin(W, C, k + 1);
      CHECK(u1 - u0 == W / C || u1 - u0 == W / C + 1);
      CHECK(fa::share_owner(W, C, u0) == k && fa::share_owner(W, C, u1 - 1) == k);
      CHECK(fa::share_owner(W, C, u0 + (u1 - u0) / 2) == k);
    }
  }
  if (failures == 0) std::printf("ok\n");
  return failures != 0;
}
