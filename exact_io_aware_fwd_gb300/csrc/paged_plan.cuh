// How the CTAs of a paged-attention launch share its keys.
//
// The work of entry b is one segment per (key/value head, row tile), each of as many key tiles
// (KT keys) as the tile's last row sees.  Laid end to end, the segments' key tiles are units
// 0 .. W - 1, and CTA c takes units [c W / C, (c + 1) W / C): equal shares whatever the lengths,
// at most two unfinished segments per CTA, so the partial results take 2 C slots however long
// the cache is.  When no segment has more than kDirectTiles key tiles, splitting would cost more
// than it gives (a join kernel has to read the parts back): then a unit is a whole segment.
// Lengths live on the device, so every CTA works this out for itself from one pass over them.
//
// A CTA takes the pieces of its share last to first.  Then the CTAs of one head's row tiles all
// start at key tile 0 of some row tile and walk the keys abreast, and so do they later in the
// tails they began with in unit order: row tiles meet the same K, V in L2 instead of reading
// them at different times.
#pragma once

#include "fa_paged.h"

namespace fa {

// Quotient of non-negative numbers; most fit 32 bits, where the division is several times shorter.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

struct Entry {
  int start, n, nc;  // first token, new tokens, and how many of them are computed
  int len;           // keys (clamped)
  int rt;            // row tiles (0: no tokens)
  int64_t tiles;     // key tiles of all its row tiles, for one key/value head
};

// Keys that row `row` (new token x group member) of an entry sees.
__device__ __forceinline__ int row_limit(const Entry& e, int causal, int G, int row) {
  return causal ? min(e.len, e.len - e.n + row / G + 1) : e.len;
}
// Key tiles of row tile r (at least one, so that a tile without keys is visited and written).
template <int R, int KT>
__device__ __forceinline__ int tiles_of(const Entry& e, int causal, int G, int r) {
  const int last = min(e.nc * G, (r + 1) * R) - 1;
  return max(1, (row_limit(e, causal, G, last) + KT - 1) / KT);
}

template <int R, int KT>
__device__ __forceinline__ Entry entry_of(const KeyList& l, const PagedArgs& a, int b, bool report) {
  Entry e;
  if (l.group_cu != nullptr) {
    int s0 = __ldg(l.group_cu + b), s1 = __ldg(l.group_cu + b + 1);
    s0 = min(max(s0, 0), a.B);
    s1 = min(max(s1, s0), a.B);
    int t0 = a.cu != nullptr ? __ldg(a.cu + s0) : s0, t1 = a.cu != nullptr ? __ldg(a.cu + s1) : s1;
    t0 = min(max(t0, 0), a.total);
    t1 = min(max(t1, t0), a.total);
    e.start = t0;
    e.n = t1 - t0;
  } else {
    token_bounds(a.cu, b, a.total, e.start, e.n);
  }
  const int64_t pages = static_cast<int64_t>(l.max_pages) << a.page_shift;
  const int cap = pages < l.max_len ? static_cast<int>(pages) : l.max_len;
  const int len = __ldg(l.lens + b);
  e.len = min(max(len, 0), cap);
  e.nc = min(e.n, l.max_q);
  if (report && (e.len != len || e.nc != e.n)) atomicCAS(a.status, 0, kErrIndex);
  e.rt = (e.nc * a.G + R - 1) / R;
  if (l.causal) {
    e.tiles = 0;
    for (int r = 0; r < e.rt; ++r) e.tiles += tiles_of<R, KT>(e, 1, a.G, r);
  } else {
    e.tiles = static_cast<int64_t>(e.rt) * max(1, (e.len + KT - 1) / KT);
  }
  return e;
}

struct Share {
  int64_t W, u0, u1;  // all units, and this CTA's
  int C;              // CTAs that have units
  bool direct;        // a unit is a whole segment
  int b;              // entry of unit u1 - 1
  int64_t off;        // its units before u1
};

// Called by all kThreads threads of the CTA.
template <int R, int KT, int kThreads, int kDirectTiles>
__device__ Share make_share(const PagedArgs& a) {
  constexpr int kWarps = kThreads / 32;
  __shared__ long long red[kWarps][2];
  __shared__ int red_max[kWarps];
  __shared__ long long at[2];
  const KeyList& l = a.list;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long seg = 0, til = 0;         // over all entries
  long long my_seg = 0, my_til = 0;   // of entry tid
  int mx = 0;
  for (int b = tid; b < l.count; b += kThreads) {
    const Entry e = entry_of<R, KT>(l, a, b, blockIdx.x == 0);
    const long long s = static_cast<long long>(e.rt) * a.Hkv, t = e.tiles * a.Hkv;
    if (b == tid) {
      my_seg = s;
      my_til = t;
    }
    seg += s;
    til += t;
    if (e.rt > 0) mx = max(mx, tiles_of<R, KT>(e, l.causal, a.G, e.rt - 1));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    seg += __shfl_xor_sync(~0u, seg, o);
    til += __shfl_xor_sync(~0u, til, o);
    mx = max(mx, __shfl_xor_sync(~0u, mx, o));
  }
  if (lane == 0) {
    red[warp][0] = seg;
    red[warp][1] = til;
    red_max[warp] = mx;
  }
  __syncthreads();
  seg = til = 0;
  mx = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    seg += red[w][0];
    til += red[w][1];
    mx = max(mx, red_max[w]);
  }
  Share sh;
  sh.direct = mx <= kDirectTiles;
  sh.W = sh.direct ? seg : til;
  // a share of fewer than kDirectTiles / 2 tiles is not worth a slot
  const long long most = sh.direct ? sh.W : (sh.W + kDirectTiles / 2 - 1) / (kDirectTiles / 2);
  sh.C = static_cast<int>(most < gridDim.x ? most : gridDim.x);
  const int c = blockIdx.x;
  sh.u0 = c < sh.C ? quotient(c * sh.W, sh.C) : 0;
  sh.u1 = c < sh.C ? quotient((c + 1) * sh.W, sh.C) : 0;
  sh.b = 0;
  sh.off = 0;
  if (sh.u0 >= sh.u1) return sh;  // uniform over the CTA
  // entry of unit u1 - 1: scan the entries kThreads at a time
  const int64_t last = sh.u1 - 1;
  long long before = 0;
  for (int b0 = 0; b0 < l.count; b0 += kThreads) {
    const int b = b0 + tid;
    long long units = sh.direct ? my_seg : my_til;
    if (b0 > 0) {
      units = 0;
      if (b < l.count) {
        const Entry e = entry_of<R, KT>(l, a, b, false);
        units = (sh.direct ? e.rt : e.tiles) * a.Hkv;
      }
    }
    long long incl = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();  // earlier readers of red are done
    if (lane == 31) red[warp][0] = incl;
    __syncthreads();
    long long pre = before, chunk = before;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) pre += red[w][0];
      chunk += red[w][0];
    }
    incl += pre;
    if (units > 0 && incl - units <= last && last < incl) {
      at[0] = b;
      at[1] = sh.u1 - (incl - units);
    }
    before = chunk;
    if (last < before) break;  // uniform
  }
  __syncthreads();
  sh.b = static_cast<int>(at[0]);
  sh.off = at[1];
  return sh;
}

// A CTA's piece of one segment: key tiles [ta, te) of row tile r for key/value head hk.
struct Piece {
  int hk, r, ta, te;
  bool whole;    // no other CTA works on the segment
  int64_t unit;  // the segment's first unit
  int tiles;     // its key tiles
};

// Walks the pieces of a CTA's share, last to first; e is the entry b of the current piece.
template <int R, int KT>
struct Walk {
  int64_t u0, u1;   // what is left of the share
  int64_t within;   // units of entry b before u1
  int b;
  bool direct;
  Entry e;

  __device__ Walk(const Share& sh, const PagedArgs& a)
      : u0(sh.u0), u1(sh.u1), within(sh.off), b(sh.b), direct(sh.direct) {
    e = entry_of<R, KT>(a.list, a, b, false);
  }
  __device__ bool next(const PagedArgs& a, Piece& p) {
    if (u0 >= u1) return false;
    while (within <= 0) {          // the entry before with tokens
      if (--b < 0) return false;   // cannot happen while u1 > 0
      e = entry_of<R, KT>(a.list, a, b, false);
      within = (direct ? e.rt : e.tiles) * a.Hkv;
    }
    const int64_t per_head = direct ? e.rt : e.tiles, x = within - 1;
    p.hk = static_cast<int>(quotient(x, per_head));
    int64_t rem = x - p.hk * per_head;
    if (direct) {
      p.r = static_cast<int>(rem);
      p.tiles = tiles_of<R, KT>(e, a.list.causal, a.G, p.r);
      p.ta = 0;
      p.te = p.tiles;
      p.whole = true;
      p.unit = --u1;
      --within;
      return true;
    }
    p.r = 0;
    p.tiles = tiles_of<R, KT>(e, a.list.causal, a.G, 0);
    while (rem >= p.tiles) {
      rem -= p.tiles;
      ++p.r;
      p.tiles = tiles_of<R, KT>(e, a.list.causal, a.G, p.r);
    }
    p.te = static_cast<int>(rem) + 1;
    p.unit = u1 - p.te;
    const int take = static_cast<int>(min(static_cast<int64_t>(p.te), u1 - u0));
    p.ta = p.te - take;
    p.whole = take == p.tiles;
    u1 -= take;
    within -= take;
    return true;
  }
};

// CTA that owns unit u: the largest c with floor(c W / C) <= u.
__device__ __forceinline__ int owner_of(const Share& sh, int64_t u) {
  return static_cast<int>(quotient((u + 1) * sh.C - 1, sh.W));
}
// (first CTA, number of CTAs) of the segment that this CTA begins.
__device__ __forceinline__ int2 span_of(const Share& sh, const Piece& p) {
  const int first = blockIdx.x;
  return make_int2(first, p.whole ? 1 : owner_of(sh, p.unit + p.tiles - 1) - first + 1);
}

}  // namespace fa
