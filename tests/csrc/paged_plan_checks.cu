// How the paged kernels' work is described, called on the host: the spans that the join reads, the
// search for a token's sequence as lane groups make it, and the shares of all workers, whose pieces
// have to be every segment's key tiles exactly once.  Prints one line per failed check.
#include <cstdint>
#include <cstdio>
#include <map>
#include <tuple>
#include <vector>

#include "fa_paged.h"
#include "paged_plan.cuh"

static int failures = 0;
#define CHECK(...) \
  do { if (!(__VA_ARGS__)) { ++failures; std::printf("line %d: %s\n", __LINE__, #__VA_ARGS__); } } while (0)

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

static unsigned seed = 12345u;
static int pick(int n) {  // 0 .. n - 1
  seed = seed * 1664525u + 1013904223u;
  return static_cast<int>((seed >> 8) % static_cast<unsigned>(n));
}

// token -> sequence for lane groups of every width, at numbers of offsets around powers of the width
template <int kLanes>
static void searches() {
  std::vector<int> sizes;
  for (int p = 1; p <= 2000; p *= kLanes)
    for (int k = -2; k <= 2; ++k)
      if (p + k >= 1 && p + k < 1200) sizes.push_back(p + k);
  sizes.insert(sizes.end(), {3, 5, 9, 17, 100, 257, 1023});
  for (int B : sizes)
    for (int most : {1, 2, 4}) {  // up to 0 (all empty), 1 and 3 tokens a sequence
      std::vector<int32_t> cu(1, pick(3));
      for (int b = 0; b < B; ++b) cu.push_back(cu.back() + pick(most));
      for (int t = -1, b = 0; t < cu[B] + 3; ++t) {
        while (b < B && cu[b + 1] <= t) ++b;
        const int want = t < cu[0] || t >= cu[B] ? -1 : b;
        CHECK(fa::token_sequence<kLanes>(cu.data(), B, t) == want);
      }
    }
}

// shares of up to 8 workers a CTA, as the few-row kernel has them
static void shares() {
  for (int C : {1, 7, 152, 153, 1000, 1215, 1216})
    for (int W : {C, C + 1, 2 * C - 1, 12345, 65537, 1 << 24, 0x7fffff00, 0x7fffffff}) {
      if (W < C) continue;
      CHECK(fa::share_begin(W, C, 0) == 0 && fa::share_begin(W, C, C) == W);
      for (int k = 0; k < C; ++k) {
        const int u0 = fa::share_begin(W, C, k), u1 = fa::share_begin(W, C, k + 1);
        CHECK(u1 - u0 == W / C || u1 - u0 == W / C + 1);
        CHECK(fa::share_owner(W, C, u0) == k && fa::share_owner(W, C, u1 - 1) == k);
      }
    }
}

// The pieces of all workers on list l.
template <int R, int KT>
static void pieces(const fa::PagedArgs& a, const fa::KeyList& l, int workers, int least, bool direct) {
  std::vector<fa::Entry> e;
  std::vector<int> first(1, 0);  // units ahead of entry b
  for (int b = 0; b < l.count; ++b) {
    e.push_back(fa::entry_of<R, KT>(l, a, b, false));
    int tiles = 0;
    for (int r = 0; r < e[b].rt; ++r) tiles += fa::tiles_of<R, KT>(e[b], l.causal, a.G, r);
    CHECK(tiles == e[b].tiles || e[b].rt == 0);
    first.push_back(first[b] + (direct ? e[b].rt : e[b].tiles) * a.Hkv);
  }
  const int W = first.back(), most = direct ? W : (W + least - 1) / least;
  const int C = most < workers ? most : workers;
  struct Part { int ta, te, worker; bool whole; int2 span; };
  std::map<std::tuple<int, int, int>, std::vector<Part>> parts;
  for (int c = 0; c < C; ++c) {
    fa::Share sh{};
    sh.W = W;
    sh.C = C;
    sh.direct = direct;
    sh.worker = c;
    sh.u0 = fa::share_begin(W, C, c);
    sh.u1 = fa::share_begin(W, C, c + 1);
    for (sh.b = 0; first[sh.b + 1] < sh.u1; ++sh.b) {}
    sh.off = sh.u1 - first[sh.b];
    sh.e = e[sh.b];
    fa::Walk<R, KT> walk(a, l, sh);
    fa::Piece p;
    int heads = 0, tails = 0;  // unfinished pieces, one slot each
    while (walk.next(a, l, p)) {
      CHECK(p.ta >= 0 && p.ta < p.te && p.te <= p.tiles && p.r >= 0 && p.r < walk.e.rt);
      CHECK(p.whole == (p.ta == 0 && p.te == p.tiles));
      if (!p.whole) (p.ta == 0 ? heads : tails)++;
      parts[{walk.b, p.hk, p.r}].push_back(
          {p.ta, p.te, c, p.whole, p.ta == 0 ? fa::span_of(sh, p) : make_int2(-1, 0)});
    }
    CHECK(heads <= 1 && tails <= 1 && walk.u0 == walk.u1);
  }
  size_t segments = 0;
  for (int b = 0; b < l.count; ++b)
    for (int hk = 0; hk < a.Hkv; ++hk)
      for (int r = 0; r < e[b].rt; ++r) {
        ++segments;
        const auto& v = parts[{b, hk, r}];  // in the order of the workers, which is the keys'
        int at = 0;
        for (size_t i = 0; i < v.size(); ++i) {
          CHECK(v[i].ta == at && v[i].worker == v[0].worker + static_cast<int>(i));
          at = v[i].te;
        }
        CHECK(at == fa::tiles_of<R, KT>(e[b], l.causal, a.G, r));
        if (v.empty()) continue;
        CHECK(v[0].span.x == v[0].worker && v[0].span.y == static_cast<int>(v.size()));
        CHECK(fa::span_ok(v[0].span.x, v[0].span.y, workers));
      }
  CHECK(parts.size() == segments);
}

static void plans() {
  for (int round = 0; round < 150; ++round) {
    const int B = 1 + pick(round % 4 == 0 ? 300 : 12), groups = 1 + pick(4);
    const int long_keys = pick(3) == 0 ? 20000 : 600, long_q = pick(3) == 0 ? 300 : 4;
    std::vector<int32_t> cu(1, 0), lens, cut, pre;
    for (int b = 0; b < B; ++b) {
      cu.push_back(cu.back() + pick(long_q));
      lens.push_back(pick(5) == 0 ? 0 : pick(long_keys));
    }
    for (int g = 0; g <= groups; ++g) cut.push_back(static_cast<int32_t>(static_cast<int64_t>(B) * g / groups));
    for (int g = 0; g < groups; ++g) pre.push_back(pick(4) == 0 ? 0 : pick(long_keys));
    fa::PagedArgs a{};
    const int heads[] = {1, 3, 4, 8, 128};
    a.cu = cu.data();
    a.B = B;
    a.total = cu.back();
    a.G = heads[pick(5)];
    a.Hkv = 1 + pick(3);
    a.H = a.G * a.Hkv;
    a.page_shift = 4;
    fa::KeyList& l = a.list[0];
    l.count = B;
    l.lens = lens.data();
    l.max_pages = 20000 / 16;
    l.max_len = pick(4) == 0 ? 500 : 20000;       // lengths past it are clamped
    l.max_q = pick(4) == 0 ? 2 : 0x7fffffff;      // tokens past it are not computed
    l.causal = pick(2);
    fa::KeyList& g = a.list[1];
    g = l;
    g.count = groups;
    g.lens = pre.data();
    g.group_cu = cut.data();
    g.max_q = 0x7fffffff;
    g.causal = 0;
    for (int li = 0; li < 2; ++li)
      for (bool direct : {false, true}) {
        pieces<fa::kPagedRows, fa::kPagedKeys>(a, a.list[li], fa::kPagedCtas * fa::kPagedWarps, 2, direct);
        pieces<fa::kPagedRows, fa::kPagedKeys>(a, a.list[li], fa::kPagedCtas, 2 * fa::kPagedWarps, direct);
        pieces<fa::kPagedMmaRows, fa::kPagedMmaKeys>(a, a.list[li], 1 + pick(fa::kPagedCtas), 2, direct);
      }
  }
}

int main() {
  spans();
  searches<2>();
  searches<8>();
  searches<16>();
  searches<32>();
  shares();
  plans();
  if (failures == 0) std::printf("ok\n");
  return failures != 0;
}
