// How the CTAs of a paged-attention launch share its keys.
//
// The work of entry b is one segment per (key/value head, row tile), each of ceil(len / KT) key
// tiles.  Laid end to end, the segments' key tiles are units 0 .. W - 1, and CTA c takes units
// [c W / C, (c + 1) W / C): equal shares whatever the lengths, at most two unfinished segments
// per CTA, so the partial results take 2 C slots however long the cache is.  When no entry has
// more than kDirectTiles key tiles, splitting would cost more than it gives (a join kernel has
// to read the parts back): then a unit is a whole segment.  Lengths live on the device, so every
// CTA works this out for itself from one pass over them.
#pragma once

#include "fa_paged.h"

namespace fa {

struct Entry {
  int start, n, nc;  // first token, new tokens, and how many of them are computed
  int len;           // keys (clamped)
  int tiles, rt;     // key tiles (at least 1) and row tiles (0: no tokens)
};

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
  e.tiles = max(1, (e.len + KT - 1) / KT);
  e.rt = (e.nc * a.G + R - 1) / R;
  return e;
}

struct Share {
  int64_t W, u0, u1;  // all units, and this CTA's
  int C;              // CTAs that have units
  bool direct;        // a unit is a whole segment
  int b;              // entry of unit u0
  int64_t off;        // its units before u0
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
  long long seg = 0, til = 0;
  int mx = 0;
  for (int b = tid; b < l.count; b += kThreads) {
    const Entry e = entry_of<R, KT>(l, a, b, blockIdx.x == 0);
    const long long s = static_cast<long long>(e.rt) * a.Hkv;
    seg += s;
    til += s * e.tiles;
    if (s > 0) mx = max(mx, e.tiles);
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
  sh.u0 = c < sh.C ? c * sh.W / sh.C : 0;
  sh.u1 = c < sh.C ? (c + 1) * sh.W / sh.C : 0;
  sh.b = 0;
  sh.off = 0;
  if (sh.u0 >= sh.u1) return sh;  // uniform over the CTA
  // entry of unit u0: scan the entries kThreads at a time
  long long before = 0;
  for (int b0 = 0; b0 < l.count; b0 += kThreads) {
    const int b = b0 + tid;
    long long units = 0;
    if (b < l.count) {
      const Entry e = entry_of<R, KT>(l, a, b, false);
      units = static_cast<long long>(e.rt) * a.Hkv * (sh.direct ? 1 : e.tiles);
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
    if (units > 0 && incl - units <= sh.u0 && sh.u0 < incl) {
      at[0] = b;
      at[1] = sh.u0 - (incl - units);
    }
    before = chunk;
    if (sh.u0 < before) break;  // uniform
  }
  __syncthreads();
  sh.b = static_cast<int>(at[0]);
  sh.off = at[1];
  return sh;
}

// CTA that owns unit u: the largest c with floor(c W / C) <= u.
__device__ __forceinline__ int owner_of(const Share& sh, int64_t u) {
  return static_cast<int>(((u + 1) * sh.C - 1) / sh.W);
}

}  // namespace fa
