// Bounds of the cache's pages, and the pages that a query attends to.
//
// A page of keys lies in the box lo_e <= k_e <= hi_e (element by element), so
//   score(q, page) = sum_e max(q_e, 0) hi_e + min(q_e, 0) lo_e
// is at least q.k for every key of the page: the cheapest score that no key of the page can beat.
// It costs two rows a page instead of page_size of them.  The page's score for a key/value head is
// the largest over its group's queries, because the group reads one list of pages.
#include <algorithm>

#include "fa_cache.h"
#include "fa_internal.h"
#include "paged_rows.cuh"
#include "select_kth.cuh"
#include "sm103.cuh"

namespace fa {

namespace {

__device__ __forceinline__ __nv_bfloat162 pair2(uint32_t u) {
  return *reinterpret_cast<__nv_bfloat162*>(&u);
}
__device__ __forceinline__ uint32_t bits2(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  return bits2(__hmin2_nan(pair2(a), pair2(b)));
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  return bits2(__hmax2_nan(pair2(a), pair2(b)));
}

// 16 bytes of global memory into shared memory, fetched from memory 256 bytes at a time; zeros where
// there are none.
__device__ __forceinline__ void fetch_once(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ uint4 from_shared(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}

// ---- the mask of a tree: a thread follows its token's parents, whose indices descend, and writes
// the words of its row from the last to the first.
constexpr int kTreeThreads = 128;

__global__ void __launch_bounds__(kTreeThreads) tree_mask_kernel(const int32_t* parents, const int32_t* cu,
                                                                 int B, int total, int words,
                                                                 uint64_t* mask, int* status) {
  begin_launch();
  const int64_t t64 = static_cast<int64_t>(blockIdx.x) * kTreeThreads + threadIdx.x;
  const int lane = threadIdx.x & 31;
  // the sequence of the warp's first token, then on from there
  const int t0 = static_cast<int>(min(t64 - lane, static_cast<int64_t>(total) - 1));
  int b = token_sequence_group<32>(cu, B, t0, lane, ~0u);
  if (t64 >= total) return;
  const int t = static_cast<int>(t64);
  if (cu == nullptr) b = t < B ? t : -1;
  else if (b < 0 && t0 < __ldg(cu)) b = 0;  // tokens before the first sequence
  if (b < 0) return;                        // behind the last sequence
  int start = 0, n = 0;
  for (; b < B; ++b) {
    token_bounds(cu, b, total, start, n);
    if (t < start + n) break;
  }
  if (b == B || t < start) return;
  int i = t - start;
  if (i >= 64LL * words) atomicCAS(status, 0, kErrIndex);  // has no bit
  uint64_t* row = mask + static_cast<int64_t>(t) * words;
  uint64_t bits = 0;
  int w = words - 1;
  while (i >= 0) {
    if (i < 64LL * words) {
      for (; w > i >> 6; --w) {
        row[w] = bits;
        bits = 0;
      }
      bits |= 1ull << (i & 63);
    }
    const int p = __ldg(parents + start + i);
    if (p < -1 || p >= i) {
      atomicCAS(status, 0, kErrIndex);
      break;
    }
    i = p;
  }
  for (; w >= 0; --w) {
    row[w] = bits;
    bits = 0;
  }
}

// ---- bounds
constexpr int kBoundThreads = 128;

// One warp a page and head: D / 8 lanes a row, eight rows a lane on the way.  Bound by reading the
// keys once: 16 prompts of 512 to 4096 tokens, 16 heads, pages of 16: 28.0 us (6.1 TB/s); one page of each of
// 64 sequences 3.9 us, which are the launch and three dependent reads.
template <int D>
__global__ void __launch_bounds__(kBoundThreads) page_bounds_kernel(const BoundsArgs a) {
  constexpr int L = D / 8, kRows = 32 / L, kAhead = 8;
  begin_launch();
  const CacheSeqs& c = a.c;
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kBoundThreads / 32) + (threadIdx.x >> 5);
  const int64_t slots = static_cast<int64_t>(c.total >> c.page_shift) + 2 * static_cast<int64_t>(c.B);
  if (unit >= slots * c.Hkv) return;
  if (unit < c.B && c.cu != nullptr && lane == 0) {  // (there are more warps than sequences)
    const int s = static_cast<int>(unit);
    if (pages_left_out(__ldg(c.cu + s), __ldg(c.cu + s + 1), c.total, keys_of(c, s, false), c.page_shift))
      atomicCAS(c.status, 0, kErrIndex);
  }
  const int slot = static_cast<int>(unit / c.Hkv), h = static_cast<int>(unit - static_cast<int64_t>(slot) * c.Hkv);
  // the last sequence whose first slot is not behind this one
  OffsetSearch s{0, c.B};
  while (true) {
    const int step = s.step(32), i = lane * step;
    const bool le = i < s.n && first_slot(c.cu, s.lo + i, c.total, c.page_shift) <= slot;
    const int hits = __popc(__ballot_sync(~0u, le));
    if (hits == 0) return;  // offsets that do not ascend
    s.narrow(step, hits);
    if (step == 1) break;
  }
  const int b = s.lo;
  int start, n;
  token_bounds(c.cu, b, c.total, start, n);
  const int i = slot - first_slot(c.cu, b, c.total, c.page_shift);
  if (i >= (n >> c.page_shift) + 2) return;  // offsets that do not ascend
  const int len = keys_of(c, b, lane == 0 && i == 0);
  const int page = (max(len - n, 0) >> c.page_shift) + i;
  const int left = len - (page << c.page_shift);  // keys from the page's first one on
  if (n == 0 || left <= 0) return;
  const int phys = page_of(c, b, page);
  if (phys < 0) return;
  const int rows = min(left, 1 << c.page_shift);
  const int64_t at = static_cast<int64_t>(phys) * c.Hkv + h;
  const uint4* src = reinterpret_cast<const uint4*>(a.k_cache + (at << c.page_shift) * D) + lane % L;
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    lo[k] = 0x7f807f80u;
    hi[k] = 0xff80ff80u;
  }
  for (int r0 = 0; r0 < rows; r0 += kRows * kAhead) {
    uint4 v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)  // past the end: the last row again
      v[k] = src[min(r0 + k * kRows + lane / L, rows - 1) * L];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      lo[0] = min2(lo[0], v[k].x); hi[0] = max2(hi[0], v[k].x);
      lo[1] = min2(lo[1], v[k].y); hi[1] = max2(hi[1], v[k].y);
      lo[2] = min2(lo[2], v[k].z); hi[2] = max2(hi[2], v[k].z);
      lo[3] = min2(lo[3], v[k].w); hi[3] = max2(hi[3], v[k].w);
    }
  }
#pragma unroll
  for (int o = L; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      lo[k] = min2(lo[k], __shfl_xor_sync(~0u, lo[k], o));
      hi[k] = max2(hi[k], __shfl_xor_sync(~0u, hi[k], o));
    }
  uint4* dst = reinterpret_cast<uint4*>(a.bounds + at * 2 * D) + lane % L;
  if (lane < L) dst[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  else if (lane < 2 * L) dst[L] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
}

// ---- scores
// A warp takes 16 pages of one key/value head as the rows of an m16n8k16 product whose columns are
// queries: [hi, lo] times [max(q, 0), min(q, 0)].  Which element of a row is which k of the product does
// not matter as long as both sides agree, so lane l % 4 takes eight neighbouring elements, 16 bytes, as
// k = 2c, 2c + 1, 2c + 8, 2c + 9 of two products, and each lane reads what it fetched itself.
// Bound by reading the bounds once.  The bytes on the way wait in shared memory, 24 warps of 8 KB an SM
// (d = 128); in registers it is 18: 18.6 us for 512 rows of up to 256 pages and their selection, cold
// caches, this 17.6, and of that this kernel takes 9; 64 sequences of 131072 keys 182 and 171 us.
// (Before that: queries as the rows, twice the products, 4% slower, all products in one chain 8%, 8
// pages a warp 25%, 32 10%; 4 warps a CTA and 2 are the same.)
constexpr int kScoreWarps = 2, kScorePages = 16, kScoreCols = 8;

// kKeep: the bounds, read by many tiles of queries, stay in registers, of which they take most (2
// sequences of 128 new tokens and 131072 keys: 190 us, from shared memory 261).
template <int D, bool kKeep>
__global__ void __launch_bounds__(32 * kScoreWarps) page_score_kernel(const SelectArgs a, int chunks) {
  constexpr int J = D / 32;  // 16-byte pieces of a lane's part of a row
  __shared__ float tile[kScoreWarps][kScorePages][kScoreCols + 1];
  __shared__ uint4 box[kScoreWarps][4 * J][32];  // what each lane fetched: lo, hi of both its pages
  begin_launch();
  const CacheSeqs& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = static_cast<int>(blockIdx.x) / chunks, chunk = static_cast<int>(blockIdx.x) % chunks;
  const int b = bh / c.Hkv, hk = bh - b * c.Hkv;
  const int p0 = (chunk * kScoreWarps + warp) * kScorePages;
  // the pages, the length and the offsets are loaded together
  int phys[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int p = p0 + 8 * t + (lane >> 2);
    phys[t] = p < c.max_pages ? __ldg(c.block_table + static_cast<int64_t>(b) * c.max_pages + p) : -1;
  }
  const int len = keys_of(c, b, threadIdx.x == 0 && chunk == 0 && hk == 0);
  int start, n;
  token_bounds(c.cu, b, c.total, start, n);
  const int pages = (len + (1 << c.page_shift) - 1) >> c.page_shift;
  if (p0 >= pages || n == 0) return;
  const uint32_t own = smem_u32(&box[warp][0][lane]);
  uint4 kept[kKeep ? 4 * J : 1];
  auto bound = [&](int t, int high, int j) {
    const int x = (t * 2 + high) * J + j;
    return kKeep ? kept[kKeep ? x : 0] : from_shared(own + x * 512);
  };
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    if (p0 + 8 * t + (lane >> 2) >= pages) {
      phys[t] = -1;
    } else if (phys[t] < 0 || phys[t] >= c.num_pages) {
      phys[t] = -1;
      atomicCAS(c.status, 0, kErrIndex);
    }
    const uint4* src = reinterpret_cast<const uint4*>(
                           a.bounds + (static_cast<int64_t>(max(phys[t], 0)) * c.Hkv + hk) * 2 * D) + (lane & 3);
#pragma unroll
    for (int x = 0; x < 2 * J; ++x)
      fetch_once(own + (t * 2 * J + x) * 512, src + x / J * (D / 8) + x % J * 4, phys[t] >= 0);
  }
  rows16::cp_commit();
  // tokens of a tile of columns, or tiles of a token
  const int per = a.G <= kScoreCols ? kScoreCols / a.G : 1, cols = min(a.G, kScoreCols);
  float* mine = &tile[warp][0][0];
  bool landed = kKeep;
  if (kKeep) {
    rows16::cp_wait<0>();  // (each lane reads what it fetched itself)
#pragma unroll
    for (int x = 0; x < 4 * J; ++x) kept[kKeep ? x : 0] = from_shared(own + x * 512);
  }
  for (int i0 = 0; i0 < n; i0 += per) {
    float best = -INFINITY;  // of page `lane` % 16, where a token has several tiles
    for (int g0 = 0; g0 < a.G; g0 += kScoreCols) {
      const int col = lane >> 2, tok = i0 + col / cols, g = g0 + col % cols;
      const bool live = col < per * cols && tok < n && g < a.G;
      const uint4* q = reinterpret_cast<const uint4*>(
                           a.q + (static_cast<int64_t>(start + (live ? tok : 0)) * a.H + hk * a.G + (live ? g : 0)) * D) +
                       (lane & 3);
      uint4 w[J];
#pragma unroll
      for (int j = 0; j < J; ++j) w[j] = live ? __ldg(q + 4 * j) : make_uint4(0u, 0u, 0u, 0u);
      if (!landed) rows16::cp_wait<0>();
      landed = true;
      float s[4] = {0.f, 0.f, 0.f, 0.f}, z[3][4] = {};  // four short chains of products
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint4 v = w[j], hi0 = bound(0, 1, j), hi1 = bound(1, 1, j), lo0 = bound(0, 0, j), lo1 = bound(1, 0, j);
        const uint32_t h0[4] = {hi0.x, hi1.x, hi0.y, hi1.y};
        const uint32_t h1[4] = {hi0.z, hi1.z, hi0.w, hi1.w};
        const uint32_t l0[4] = {lo0.x, lo1.x, lo0.y, lo1.y};
        const uint32_t l1[4] = {lo0.z, lo1.z, lo0.w, lo1.w};
        rows16::mma16816(s, h0, max2(v.x, 0u), max2(v.y, 0u));
        rows16::mma16816(z[0], l0, min2(v.x, 0u), min2(v.y, 0u));
        rows16::mma16816(z[1], h1, max2(v.z, 0u), max2(v.w, 0u));
        rows16::mma16816(z[2], l1, min2(v.z, 0u), min2(v.w, 0u));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] = (s[k] + z[1][k]) + (z[0][k] + z[2][k]);
      __syncwarp();  // the last tile has been read
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = (lane >> 2) + 8 * (k >> 1), at = (lane & 3) * 2 + (k & 1);
        // a score that is not a number counts as infinity
        mine[row * (kScoreCols + 1) + at] = s[k] == s[k] ? s[k] : INFINITY;
      }
      __syncwarp();
      for (int o = lane; o < per * kScorePages; o += 32) {
        const int tt = o / kScorePages, page = o % kScorePages, here = min(cols, a.G - g0);
        float m = -INFINITY;
        for (int x = 0; x < here; ++x) m = fmaxf(m, mine[page * (kScoreCols + 1) + tt * cols + x]);
        if (a.G > kScoreCols) {
          m = best = fmaxf(best, m);
          if (g0 + kScoreCols < a.G) continue;
        }
        if (i0 + tt < n && p0 + page < pages)
          a.score[(static_cast<int64_t>(start + i0 + tt) * c.Hkv + hk) * a.max_pages + p0 + page] = m;
      }
    }
  }
  uint32_t most = 0;  // largest |bound| (NaN, if one is)
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint4 lo = bound(t, 0, j), hi = bound(t, 1, j);
      const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) most = bits2(__hmax2_nan(pair2(most), __habs2(pair2(u[k]))));
    }
  most = max(most & 0x7fffu, most >> 16 & 0x7fffu);  // as bits: NaN is above infinity
  most = __reduce_max_sync(~0u, most);
  if (lane == 0)
    a.reach[static_cast<int64_t>(bh) * ((a.max_pages + kScorePages - 1) / kScorePages) + p0 / kScorePages] =
        __uint_as_float(most << 16);
}

// ---- selection
// One CTA a token and key/value head.  A page is in or out by a comparison, so the choice is that of
// exact scores: the float32 scores above are off by at most delta = 2^-15 sum_e |q_e| max |bound|
// (16 products of 16 terms each, every addition off by at most 2^-23 of what has been added up so
// far in magnitude).  With t the k-th largest of them, every page more than 2 delta above t is in and
// every page more than 2 delta below it is out; the few between are scored again as exactly as in 64
// bits.
constexpr int kBorder = 512;  // pages next to the border that are ranked in shared memory
constexpr int kFew = 16;      // few enough to be taken for the border without another pass

// What a warp needs of a page and the queries: E elements a lane, of kHeads heads at a time.
constexpr int kFineHeads = 4;
template <int D>
struct FineRows {
  const __nv_bfloat16 *box, *q;
  bool there;  // a page outside the pool has bounds of 0
  __device__ FineRows(const SelectArgs& a, int b, int hk, int t, int p, int lane) {
    const int phys = page_of(a.c, b, p);
    there = phys >= 0;
    box = a.bounds + (static_cast<int64_t>(max(phys, 0)) * a.c.Hkv + hk) * 2 * D + lane * (D / 32);
    q = a.q + (static_cast<int64_t>(t) * a.H + hk * a.G) * D + lane * (D / 32);
  }
};

// A power of two, as two factors that are applied one after the other: what scales a number below the
// smallest normal one to about 1 is no float.
struct Scale {
  float pre, by;
  __device__ float operator()(float x) const { return x * pre * by; }
};
// x > 0 to [1/2, 1) (x < 2^126; 0: anything).
__device__ __forceinline__ Scale scale_to_one(float x) {
  const float pre = x < 0x1p-126f ? 0x1p64f : 1.f;
  const int e = static_cast<int>(__float_as_uint(x * pre) >> 23);  // x pre < 2^(e - 126)
  return {pre, x == 0.f ? 1.f : __uint_as_float(static_cast<uint32_t>(max(253 - e, 1)) << 23)};
}

// The score as an integer: sum q_e box_e in units of 2^-62, where S = sum |q_e| max |bound| has been
// scaled to [1/2, 1) by powers of two (S may be off by its float32 sum, 2^-19 of it).  The products u_e
// are exact and below 1.  Their next 22, 23 and 23 bits are taken off as integers one after the other
// (adding 3/2 2^23 rounds to one; what is left is at most half of the last one's unit, so the next are
// at most 2^22), and the integers are added up, in any order.  D products rounded at 2^-69 are off by
// 2^-62 together, cutting the sum to units of 2^-62 by less than that: of two scores that are 3 2^-62,
// below 2^-59 S, apart or more, the larger one stays the larger.  fp64 would do, but at two
// multiply-adds a cycle and SM it made this the longest part of the kernel (18 us of 33).
template <int D>
__device__ __forceinline__ int64_t fine_score(const SelectArgs& a, int b, int hk, int t, int p, int lane,
                                              Scale q_scale, Scale box_scale) {
  constexpr int E = D / 32;
  constexpr float kRound = 12582912.f;  // 3/2 2^23
  const FineRows<D> r(a, b, hk, t, p, lane);
  float lo[E], hi[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    lo[e] = r.there ? box_scale(__bfloat162float(r.box[e])) : 0.f;
    hi[e] = r.there ? box_scale(__bfloat162float(r.box[D + e])) : 0.f;
  }
  int64_t best = INT64_MIN;
  for (int g = 0; g < a.G; g += kFineHeads) {
    uint32_t sum[kFineHeads][3];
#pragma unroll
    for (int i = 0; i < kFineHeads; ++i) {
      sum[i][0] = sum[i][1] = sum[i][2] = 0u;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float q = q_scale(__bfloat162float(r.q[min(g + i, a.G - 1) * D + e]));
        float u = q * (q > 0.f ? hi[e] : lo[e]), t;
        t = fmaf(u, 0x1p22f, kRound);
        u = fmaf(t - kRound, -0x1p-22f, u);
        sum[i][0] += __float_as_uint(t) - __float_as_uint(kRound);
        t = fmaf(u, 0x1p45f, kRound);
        u = fmaf(t - kRound, -0x1p-45f, u);
        sum[i][1] += __float_as_uint(t) - __float_as_uint(kRound);
        t = fmaf(u, 0x1p68f, kRound);
        sum[i][2] += __float_as_uint(t) - __float_as_uint(kRound);
      }
    }
#pragma unroll
    for (int i = 0; i < kFineHeads; ++i) {
      const int s0 = __reduce_add_sync(~0u, static_cast<int>(sum[i][0]));
      const int s1 = __reduce_add_sync(~0u, static_cast<int>(sum[i][1]));
      const int s2 = __reduce_add_sync(~0u, static_cast<int>(sum[i][2]));
      const int64_t x = (((static_cast<int64_t>(s0) << 23) + s1) << 17) + (s2 >> 6);
      best = x > best ? x : best;
    }
  }
  return best;
}

// In 64 bits, where something is not finite or S or one of its factors is 2^126 or more (sums of products
// that are exact, off by 2^-49 S).
template <int D>
__device__ __forceinline__ double odd_score(const SelectArgs& a, int b, int hk, int t, int p, int lane) {
  constexpr int E = D / 32;
  const FineRows<D> r(a, b, hk, t, p, lane);
  double best = -INFINITY;
  for (int g = 0; g < a.G; ++g) {
    double x = 0.0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const double v = static_cast<double>(__bfloat162float(r.q[g * D + e]));
      const double lo = r.there ? static_cast<double>(__bfloat162float(r.box[e])) : 0.0;
      const double hi = r.there ? static_cast<double>(__bfloat162float(r.box[D + e])) : 0.0;
      x += (v < 0.0 ? 0.0 : v) * hi + (v > 0.0 ? 0.0 : v) * lo;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    if (x != x) x = INFINITY;
    best = x > best ? x : best;
  }
  return best;
}
// The largest sum |q_e| of heads g0, g0 + step, ... of a group (infinite where one is not a number).
template <int D>
__device__ __forceinline__ float query_size(const SelectArgs& a, int t, int hk, int g0, int step, int lane) {
  const __nv_bfloat16* q = a.q + (static_cast<int64_t>(t) * a.H + hk * a.G) * D + lane;
  float size = 0.f;
#pragma unroll 4
  for (int g = g0; g < a.G; g += step) {
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < D; e += 32) x += fabsf(__bfloat162float(q[g * D + e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    size = x == x ? fmaxf(size, x) : INFINITY;
  }
  return size;
}
// The pages with keys that token t sees (-1: behind the last sequence), and its sequence; by whole
// warps.
__device__ __forceinline__ int visible_pages(const SelectArgs& a, int t, int& b, int lane, bool first, bool head0) {
  const CacheSeqs& c = a.c;
  b = token_sequence_group<32>(c.cu, c.B, t, lane, ~0u);
  if (b < 0) return -1;
  int start, n;
  token_bounds(c.cu, b, c.total, start, n);
  if (t < start || t >= start + n) {  // offsets that do not ascend
    if (first) atomicCAS(c.status, 0, kErrIndex);
    return -1;
  }
  const int len = keys_of(c, b, head0 && first);
  const int sees = min(max(len - n + (t - start) + 1, 0), len);
  return (sees + (1 << c.page_shift) - 1) >> c.page_shift;
}

// kSelectRounds: scores of a thread in registers; further ones are read again.  (A warp a row that closes
// in on the k-th by votes, without a barrier: 21.6 us instead of 16.7 for 512 rows of up to 256 pages in L2.)
constexpr float kMost = 3.402823466e38f;

// behind_scores: page_score_kernel is the kernel ahead, so what it did not write is complete.
template <int D, int kSelectThreads, int kSelectRounds>
__global__ void __launch_bounds__(kSelectThreads) select_pages_kernel(const SelectArgs a, const bool behind_scores) {
  constexpr int kWarps = kSelectThreads / 32, kHeld = kSelectRounds * kSelectThreads;
  __shared__ union {
    KthShared<kSelectThreads, uint32_t> k32;
    KthShared<kSelectThreads, uint64_t> k64;
    struct {
      uint64_t value[kBorder];
      int page[kBorder];
      bool take[kBorder];
    } border;
  } sh;
  __shared__ OrderShared<kSelectThreads, kSelectRounds> order_sh;
  __shared__ float red[2][kWarps];
  __shared__ int counts[kWarps], border_count;
  let_next_launch();
  if (!behind_scores) wait_for_last_launch();
  const CacheSeqs& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.x / c.Hkv, hk = blockIdx.x - t * c.Hkv;
  // (loaded while the token's sequence is searched for)
  float size = behind_scores ? query_size<D>(a, t, hk, warp, kWarps, lane) : 0.f;
  int b;
  const int pages = visible_pages(a, t, b, lane, tid == 0, hk == 0);
  const int mid = pages - a.first - a.last, k = a.top - a.first - a.last;  // k of the pages in between
  int32_t* out = a.pages + static_cast<int64_t>(blockIdx.x) * a.top;
  if (behind_scores) wait_for_last_launch();
  if (pages < 0) return;  // behind the last sequence
  if (pages <= a.top) {
    for (int i = tid; i < a.top; i += kSelectThreads) out[i] = i < pages ? i : -1;
    return;
  }
  for (int i = tid; i < a.first; i += kSelectThreads) out[i] = i;
  for (int i = tid; i < a.last; i += kSelectThreads) out[a.top - a.last + i] = pages - a.last + i;
  if (k == 0) return;
  float* score = a.score + static_cast<int64_t>(blockIdx.x) * a.max_pages + a.first;
  float x[kSelectRounds];
#pragma unroll
  for (int i = 0; i < kSelectRounds; ++i) {
    const int at = i * kSelectThreads + tid;
    x[i] = at < mid ? score[at] : 0.f;
  }
  // delta
  const float* reach = a.reach + (static_cast<int64_t>(b) * c.Hkv + hk) * ((a.max_pages + kScorePages - 1) / kScorePages);
  float far = 0.f;
  for (int i = tid; i < (pages + kScorePages - 1) / kScorePages; i += kSelectThreads) {
    const float r = reach[i];
    far = r == r ? fmaxf(far, r) : INFINITY;
  }
  far = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(far)));  // (none is negative)
  if (lane == 0) {
    red[0][warp] = far;
    red[1][warp] = size;
  }
  if (tid == 0) border_count = 0;
  __syncthreads();
  far = __uint_as_float(__reduce_max_sync(~0u, lane < kWarps ? __float_as_uint(red[0][lane]) : 0u));
  size = __uint_as_float(__reduce_max_sync(~0u, lane < kWarps ? __float_as_uint(red[1][lane]) : 0u));
  // (what is added: sums below the smallest normal number have no such relative error)
  const float delta = fmaf(far * size, 0x1p-15f, 0x1p-117f);
  // something is not finite, too large to be scaled below 1, or so large that a score with 2 delta
  // added might not be finite: every score in 64 bits
  const bool odd = !(far * size < 0x1p126f && far < 0x1p126f && size < 0x1p126f);

  float above = kMost, below = -INFINITY;  // in, and at least in question
  if (!odd) {
    auto each = [&](auto f) {
#pragma unroll
      for (int i = 0; i < kSelectRounds; ++i)
        if (i * kSelectThreads + tid < mid) f(ordered(x[i]));
      for (int at = kHeld + tid; at < mid; at += kSelectThreads) f(ordered(score[at]));
    };
    const Kth<uint32_t> kth = kth_largest<kSelectThreads, false, uint32_t>(k, kFew, each, sh.k32);
    above = unordered(kth.base + kth.range) + 2.f * delta;
    below = unordered(kth.base) - 2.f * delta;
    __syncthreads();  // the bins are free
  }
  // page i's score exactly, as a number that orders like it
  const Scale q_scale = scale_to_one(size);
  Scale box_scale = scale_to_one(far);
  if (q_scale(size) * box_scale(far) < 0.5f) box_scale.by *= 2.f;
  auto exact = [&](int i) {
    return odd ? ordered(odd_score<D>(a, b, hk, t, a.first + i, lane))
               : static_cast<uint64_t>(fine_score<D>(a, b, hk, t, a.first + i, lane, q_scale, box_scale)) ^ (1ull << 63);
  };
  // a score next to the border is replaced by its number in the list, as the bits of a NaN
  auto held = [](int at) { return __int_as_float(0x7fc00000 | at); };
  int sure = 0;
  auto classify = [&](float& v, int at) {
    if (!odd && v > above) {
      ++sure;
    } else if (odd || v >= below) {
      const int e = atomicAdd(&border_count, 1);
      if (e < kBorder) {
        sh.border.page[e] = at;
        v = held(e);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kSelectRounds; ++i)
    if (i * kSelectThreads + tid < mid) classify(x[i], i * kSelectThreads + tid);
  for (int at = kHeld + tid; at < mid; at += kSelectThreads) {
    float v = score[at];
    classify(v, at);
  }
  sure = __reduce_add_sync(~0u, sure);
  if (lane == 0) counts[warp] = sure;
  __syncthreads();
  sure = __reduce_add_sync(~0u, lane < kWarps ? counts[lane] : 0);
  const int border = border_count, need = k - sure;  // need <= border
  if (border <= kBorder) {
    if (need < border) {
      for (int e = warp; e < border; e += kWarps) {
        const uint64_t v = exact(sh.border.page[e]);
        if (lane == 0) sh.border.value[e] = v;
      }
      __syncthreads();
    }
    for (int e = tid; e < border; e += kSelectThreads) {
      const uint64_t v = sh.border.value[e];
      const int p = sh.border.page[e];
      int rank = 0;
      if (need < border)
        for (int j = 0; j < border; ++j) {
          const uint64_t y = sh.border.value[j];
          rank += y > v || (y == v && sh.border.page[j] < p);
        }
      sh.border.take[e] = rank < need;
      if (p >= kHeld) score[p] = rank < need ? INFINITY : -INFINITY;
    }
    __syncthreads();
  } else {
    // many equal or nearly equal pages, or something that is not finite: through memory
    uint64_t* fine = a.fine + static_cast<int64_t>(blockIdx.x) * a.max_pages + a.first;
    auto here = [&](float v) { return odd || !(v > above || v < below); };
    for (int i = warp; i < mid; i += kWarps) {
      if (!here(score[i])) continue;
      const uint64_t y = exact(i);
      if (lane == 0) fine[i] = y;
    }
    __syncthreads();
    auto each = [&](auto f) {
      for (int i = tid; i < mid; i += kSelectThreads)
        if (here(score[i])) f(fine[i]);
    };
    const Kth<uint64_t> kth = kth_largest<kSelectThreads, false, uint64_t>(need, 0, each, sh.k64);
    // in order, so that of equal ones the first are taken
    int taken = 0;
    for (int i0 = 0; i0 < mid; i0 += kSelectThreads) {
      const int i = i0 + tid;
      const bool in = i < mid && here(score[i]);
      const uint64_t key = in ? fine[i] : 0;
      const bool tie = in && kth.holds(key);
      const unsigned ties = __ballot_sync(~0u, tie);
      if (lane == 0) counts[warp] = __popc(ties);
      __syncthreads();
      int before = taken + __popc(ties & ((1u << lane) - 1u));
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += counts[w];
        taken += counts[w];
      }
      if (in) score[i] = (tie ? before < kth.need : kth.under(key)) ? INFINITY : -INFINITY;
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kSelectRounds; ++i)
      if (i * kSelectThreads + tid < mid) x[i] = score[i * kSelectThreads + tid];
  }
  // the pages in order
  Order<kSelectThreads, kSelectRounds> order{order_sh};
  int done = a.first;
  for (int r0 = 0; r0 < mid; r0 += kHeld) {
    if (r0 > 0) {
#pragma unroll
      for (int i = 0; i < kSelectRounds; ++i) {
        const int at = r0 + i * kSelectThreads + tid;
        x[i] = at < mid ? score[at] : 0.f;
      }
    }
    auto in = [&](int i) {
      if (r0 + i * kSelectThreads + tid >= mid) return false;
      const unsigned u = __float_as_uint(x[i]);
      if (u - 0x7fc00000u < static_cast<unsigned>(kBorder)) return sh.border.take[u - 0x7fc00000u];
      return x[i] > above;
    };
    auto no = [](int) { return false; };
    const unsigned total = order.scan(in, no);
#pragma unroll
    for (int i = 0; i < kSelectRounds; ++i) {
      const bool hit = order.over(i);
      const int to = done + static_cast<int>(order.before(i));
      if (hit && to < a.top - a.last) out[to] = a.first + r0 + i * kSelectThreads + tid;  // always, while inputs stay
    }
    done += static_cast<int>(total);
    __syncthreads();
  }
}

template <int D>
cudaError_t launch_select_d(const SelectArgs& a, cudaStream_t s) {
  const int chunks = (a.max_pages + kScoreWarps * kScorePages - 1) / (kScoreWarps * kScorePages);
  const unsigned grid = static_cast<unsigned>(a.c.B) * static_cast<unsigned>(a.c.Hkv) * static_cast<unsigned>(chunks);
  const bool scores = a.max_pages > a.top && a.top > a.first + a.last;  // else nobody chooses
  if (scores) {
    // more queries of a sequence than one tile has
    const bool many = static_cast<int64_t>(a.c.total) * a.G > static_cast<int64_t>(a.c.B) * std::max(kScoreCols, a.G);
    const cudaError_t e = many ? launch_chained(page_score_kernel<D, true>, grid, 32 * kScoreWarps, 0, s, a, chunks)
                               : launch_chained(page_score_kernel<D, false>, grid, 32 * kScoreWarps, 0, s, a, chunks);
    if (e != cudaSuccess) return e;
  }
  const unsigned rows = static_cast<unsigned>(a.c.total) * static_cast<unsigned>(a.c.Hkv);
  return a.max_pages <= 4 * 256 ? launch_chained(select_pages_kernel<D, 256, 4>, rows, 256, 0, s, a, scores)
                                : launch_chained(select_pages_kernel<D, 512, 8>, rows, 512, 0, s, a, scores);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_tree_mask(const int32_t* parents, const int32_t* cu, int B, int total, int words,
                             uint64_t* mask, int* status, cudaStream_t s) {
  const unsigned grid = (static_cast<unsigned>(total) + kTreeThreads - 1) / kTreeThreads;
  return launch_chained(tree_mask_kernel, grid, kTreeThreads, 0, s, parents, cu, B, total, words, mask, status);
}

cudaError_t launch_page_bounds(int d, const BoundsArgs& a, cudaStream_t s) {
  const int64_t units = ((static_cast<int64_t>(a.c.total) >> a.c.page_shift) + 2 * static_cast<int64_t>(a.c.B)) * a.c.Hkv;
  const unsigned grid = static_cast<unsigned>((units + kBoundThreads / 32 - 1) / (kBoundThreads / 32));
  return d == 64 ? launch_chained(page_bounds_kernel<64>, grid, kBoundThreads, 0, s, a)
                 : launch_chained(page_bounds_kernel<128>, grid, kBoundThreads, 0, s, a);
}

SelectWorkspace select_workspace(int B, int total, int Hkv, int max_pages) {
  SelectWorkspace w{};
  const size_t rows = static_cast<size_t>(total) * static_cast<size_t>(Hkv), P = static_cast<size_t>(max_pages);
  w.score = 0;
  w.fine = up256(rows * P * 4);
  w.reach = w.fine + up256(rows * P * 8);
  w.total = w.reach + up256(static_cast<size_t>(B) * static_cast<size_t>(Hkv) * ((P + 15) / 16) * 4);
  return w;
}

cudaError_t launch_select_pages(int d, const SelectArgs& a, cudaStream_t s) {
  return d == 64 ? launch_select_d<64>(a, s) : launch_select_d<128>(a, s);
}

}  // namespace fa
