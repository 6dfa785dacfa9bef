// How the cache's operators divide their work, on the host.  The places that fa_page_bounds gives to the
// pages of a ragged batch: every page that holds a new key has one, no two share one, all lie in the
// launch, and the search finds each place's sequence; and which totals leave pages out.  The pieces of fa_kv_weights' workers: every key
// tile of every sequence that has queries is in one, and no more.  Prints one line per failed check.
#include <cstdio>
#include <map>
#include <tuple>
#include <vector>

#include "fa_cache.h"
#include "paged_plan.cuh"

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

// The pieces of all workers, as weights_kernel takes them.
static void pieces(const fa::PagedArgs& a, int workers) {
  constexpr int R = 1 << 30, KT = 128;
  const fa::KeyList& l = a.list[0];
  std::vector<fa::Entry> e;
  std::vector<int> first(1, 0);  // units ahead of entry b
  for (int b = 0; b < l.count; ++b) {
    e.push_back(fa::entry_of<R, KT>(l, a, b, false));
    CHECK(e[b].rt <= 1);
    first.push_back(first[b] + e[b].tiles * a.Hkv);
  }
  const int W = first.back(), C = (W + 1) / 2 < workers ? (W + 1) / 2 : workers;
  std::map<std::tuple<int, int, int>, int> seen;
  for (int c = 0; c < C; ++c) {
    fa::Share sh{};
    sh.W = W;
    sh.C = C;
    sh.worker = c;
    sh.u0 = fa::share_begin(W, C, c);
    sh.u1 = fa::share_begin(W, C, c + 1);
    for (sh.b = 0; first[sh.b + 1] < sh.u1; ++sh.b) {}
    sh.off = sh.u1 - first[sh.b];
    sh.e = e[sh.b];
    fa::Walk<R, KT> walk(a, l, sh);
    fa::Piece p;
    while (walk.next(a, l, p)) {
      CHECK(p.r == 0 && p.ta >= 0 && p.ta < p.te);
      const int tiles = (walk.e.len + KT - 1) / KT;
      for (int t = p.ta; t < (p.te < tiles ? p.te : tiles); ++t) ++seen[{walk.b, p.hk, t}];
    }
    CHECK(walk.u0 == walk.u1);
  }
  size_t all = 0;
  for (int b = 0; b < l.count; ++b)
    if (e[b].nc > 0) all += static_cast<size_t>((e[b].len + KT - 1) / KT) * static_cast<size_t>(a.Hkv);
  CHECK(seen.size() == all);
  for (const auto& s : seen) CHECK(s.second == 1);
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
        // pages of the last n keys, all counted and with a total that cuts some off
        const int cut = random(total + 2);
        int s0, some;
        fa::clamp_tokens(start, start + n, cut, s0, some);
        bool out = false;
        for (int key = len > n ? len - n : 0; key < len; ++key) {
          bool renewed = false;
          for (int k = len > some ? len - some : 0; k < len; ++k) renewed = renewed || k >> shift == key >> shift;
          out = out || !renewed;
        }
        CHECK(fa::pages_left_out(start, start + n, cut, len, shift) == out);
        CHECK(fa::pages_left_out(-1, n, total, len, shift) && fa::pages_left_out(n + 1, n, n + 1, len, shift));
      }
    }
  for (int round = 0; round < 300; ++round) {
    const int B = 1 + random(round % 5 == 0 ? 200 : 10), long_keys = random(3) == 0 ? 30000 : 700;
    std::vector<int32_t> cu(1, 0), lens;
    for (int b = 0; b < B; ++b) {
      cu.push_back(cu.back() + (random(3) == 0 ? random(200) : random(3)));
      lens.push_back(random(5) == 0 ? 0 : random(long_keys));
    }
    fa::PagedArgs a{};
    a.cu = cu.data();
    a.B = B;
    a.total = cu.back();
    a.G = 1 + random(8);
    a.Hkv = 1 + random(8);
    a.page_shift = 4;
    fa::KeyList& l = a.list[0];
    l.count = B;
    l.lens = lens.data();
    l.max_pages = 2000;
    l.max_len = random(4) == 0 ? 500 : 32000;
    l.extra = random(3);
    l.max_q = random(4) == 0 ? 2 : 0x7fffffff;
    for (int workers : {1, 1 + random(152), 152}) pieces(a, workers);
    // an entry's units are those of its row tiles, of sequences and of tokens alone
    fa::KeyList tokens = l;
    tokens.lens = nullptr;
    for (const fa::KeyList& x : {l, tokens})
      for (int causal : {0, 1}) {
        fa::KeyList y = x;
        y.causal = causal && x.lens != nullptr;
        const int b = random(B);
        const fa::Entry e = fa::entry_of<16, 16>(y, a, b, false);
        int units = 0;
        for (int r = 0; r < e.rt; ++r) units += fa::units_of<16, 16>(y, e, a.G, r);
        CHECK(e.tiles == units);
      }
  }
  std::printf(failures == 0 ? "ok\n" : "%d failures\n", failures);
  return failures == 0 ? 0 : 1;
}
