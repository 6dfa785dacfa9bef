// How the workers of a paged-attention launch share the keys of a list (a worker: a CTA of the
// tensor-core kernel or, where segments are few, of the other one, else a warp of that).
//
// The work of entry b is one segment per (key/value head, row tile), each of as many key tiles
// (KT keys) as the tile's last row sees.  Laid end to end, the segments' key tiles are units
// 0 .. W - 1, and worker c of C takes units [c W / C, (c + 1) W / C): equal shares whatever the
// lengths, at most two unfinished segments per worker, so the partial results take 2 C slots
// however long the cache is.  When no segment has more than `unsplit` key tiles, splitting
// would cost more than it gives (a join kernel has to read the parts back): then a unit is a
// whole segment.  Lengths live on the device, so every CTA works this out for itself from one
// pass over them.  Units fit 32 bits (the host refuses more).
//
// A worker takes the pieces of its share last to first.  Then the CTAs of one head's row tiles
// all start at key tile 0 of some row tile and walk the keys abreast, and so do they later in the
// tails they began with in unit order: row tiles meet the same K, V in L2 instead of reading
// them at different times.
#pragma once

#include "fa_paged.h"

namespace fa {

// Reads the launch's arguments while the kernel ahead still runs: they are in the constant cache
// when they are needed.
__device__ __forceinline__ void touch(const PagedArgs& a) {
  asm volatile("" ::"r"(a.B), "r"(a.list[0].count), "l"(a.list[0].group_cu), "l"(a.list[1].lens),
               "r"(a.list[1].causal), "l"(a.part[0].spans), "l"(a.part[1].slots),
               "l"(a.rowbuf[0]), "l"(a.status));
}

// (The functions that say how work is cut are compiled for the host as well, where they are tested:
// every key tile of every segment is some worker's, once.)
__host__ __device__ __forceinline__ int device_load(const int32_t* p) {
#ifdef __CUDA_ARCH__
  return __ldg(p);
#else
  return *p;
#endif
}

struct Entry {
  int start, n, nc;  // first token, new tokens, and how many of them are computed
  int len;           // keys (clamped)
  int rt;            // row tiles (0: no tokens)
  int tiles;         // key tiles of all its row tiles, for one key/value head
};

// Keys that row `row` (new token x group member) of an entry sees.
__host__ __device__ __forceinline__ int row_limit(const Entry& e, int causal, int G, int row) {
  return causal ? min(e.len, e.len - e.n + row / G + 1) : e.len;
}
// Key tiles of row tile r (at least one, so that a tile without keys is visited and written).
template <int R, int KT>
__host__ __device__ __forceinline__ int tiles_of(const Entry& e, int causal, int G, int r) {
  const int last = min(e.nc * G, (r + 1) * R) - 1;
  return max(1, (row_limit(e, causal, G, last) + KT - 1) / KT);
}

template <int R, int KT>
__host__ __device__ __forceinline__ Entry entry_of(const KeyList& l, const PagedArgs& a, int b,
                                                   bool report) {
  Entry e;
  const int len = device_load(l.lens + b);  // ahead of the branches: one wait for all of the loads
  bool ok;
  if (l.group_cu != nullptr) {
    const int g0 = device_load(l.group_cu + b), g1 = device_load(l.group_cu + b + 1);
    const int s0 = min(max(g0, 0), a.B), s1 = min(max(g1, s0), a.B);
    const int t0 = a.cu != nullptr ? device_load(a.cu + s0) : s0;
    const int t1 = a.cu != nullptr ? device_load(a.cu + s1) : s1;
    ok = (g0 >= 0) & (g0 <= g1) & (g1 <= a.B);
    clamp_tokens(t0, t1, a.total, e.start, e.n);
  } else {
    const int t0 = a.cu != nullptr ? device_load(a.cu + b) : b;
    const int t1 = a.cu != nullptr ? device_load(a.cu + b + 1) : b + 1;
    ok = (t0 >= 0) & (t0 <= t1) & (t1 <= a.total);
    clamp_tokens(t0, t1, a.total, e.start, e.n);
  }
  const int64_t pages = static_cast<int64_t>(l.max_pages) << a.page_shift;
  const int cap = pages < l.max_len ? static_cast<int>(pages) : l.max_len;
  e.len = min(max(len, 0), cap);
  e.nc = min(e.n, l.max_q);
#ifdef __CUDA_ARCH__
  if (report && (!ok || e.len != len || e.nc != e.n)) atomicCAS(a.status, 0, kErrIndex);
#endif
  e.rt = (e.nc * a.G + R - 1) / R;
  if (l.causal && e.n > 1) {
    e.tiles = 0;
    for (int r = 0; r < e.rt; ++r) e.tiles += tiles_of<R, KT>(e, 1, a.G, r);
  } else {
    e.tiles = e.rt * max(1, (e.len + KT - 1) / KT);
  }
  return e;
}

// Splitting W units over C workers: worker c takes [c W / C, (c + 1) W / C).  (The longer shares
// are spread over the workers on purpose: with all of them first, the CTAs of a tensor-core launch
// run in lockstep and their bursts of copies slow the MMAs: 249 instead of 226 us for 2 x 512
// tokens over 16384 keys.)  c W / C = c (W div C) + c (W mod C) / C: 32-bit divisions, C < 2^16.
__host__ __device__ inline int share_begin(int W, int C, int c) {
  const unsigned w = W, n = C, i = c;
  return static_cast<int>(i * (w / n) + i * (w % n) / n);
}
// Worker that owns unit u: the largest c with c W / C <= u.
__host__ __device__ inline int share_owner(int W, int C, int u) {
  return static_cast<int>(((static_cast<int64_t>(u) + 1) * C - 1) / W);
}

struct Share {
  int W, C;       // all units, and the workers that have some
  bool direct;    // a unit is a whole segment
  int worker;     // this worker and its units (none: u0 == u1)
  int u0, u1;
  int b, off;     // entry of unit u1 - 1, and its units before u1; -1: none (offsets that
                  // overlap, whose units do not fit 32 bits)
  Entry e;        // that entry
};

// What a list's entries add up to; red: the warps' sums in shared memory.
struct Totals {
  int seg, til, mx;  // segments, key tiles, the most of a segment
};
template <int R, int KT, int kThreads>
__device__ __forceinline__ void sum_entries(const PagedArgs& a, const KeyList& l, Entry& mine,
                                            int (*red)[kThreads / 32]) {
  const int tid = threadIdx.x;
  int seg = 0, til = 0, mx = 0;
  mine = Entry{};  // entry tid
  for (int b = tid; b < l.count; b += kThreads) {
    const Entry e = entry_of<R, KT>(l, a, b, blockIdx.x == 0);
    if (b == tid) mine = e;
    seg += e.rt * a.Hkv;
    til += e.tiles * a.Hkv;
    if (e.rt > 0) mx = max(mx, tiles_of<R, KT>(e, l.causal, a.G, e.rt - 1));
  }
  seg = __reduce_add_sync(~0u, seg);
  til = __reduce_add_sync(~0u, til);
  mx = __reduce_max_sync(~0u, mx);
  if ((tid & 31) == 0) {
    red[0][tid >> 5] = seg;
    red[1][tid >> 5] = til;
    red[2][tid >> 5] = mx;
  }
}
template <int kWarps>
__device__ __forceinline__ Totals totals_of(const int (*red)[kWarps]) {
  Totals t{0, 0, 0};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    t.seg += red[0][w];
    t.til += red[1][w];
    t.mx = max(t.mx, red[2][w]);
  }
  return t;
}

// The shares of the kWorkers workers of CTA `cta` of the `ctas` that work on list l (worker w of
// CTA c is number c + w x ctas: the first units go to different SMs), from the list's totals and
// this thread's entry.  Called by all kThreads threads; `shares` in shared memory is complete when
// it returns.
template <int R, int KT, int kThreads, int kWorkers>
__device__ __forceinline__ void share_list(const PagedArgs& a, const KeyList& l, const Totals& t,
                                           Entry mine, int cta, int ctas, int* scan,
                                           Share* shares) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool direct = t.mx <= l.unsplit;
  const int W = direct ? t.seg : t.til;
  // shares of one tile are not worth their slots (one sequence of 1000 keys and 8 heads takes 10.1
  // us either way; shares of at least four take 11.5 us, of eight 13.4)
  // (a CTA as the worker of the few-row kernel: two tiles a warp)
  constexpr int kMin = KT == kPagedKeys && kWorkers == 1 ? 2 * kPagedWarps : 2;
  const int most = direct ? W : (W + kMin - 1) / kMin;
  const int C = min(most, ctas * kWorkers);
  if (tid < kWorkers) {
    Share& s = shares[tid];
    const int c = cta + tid * ctas;
    s.W = W;
    s.C = C;
    s.direct = direct;
    s.worker = c;
    s.u0 = c < C ? share_begin(W, C, c) : 0;
    s.u1 = c < C ? share_begin(W, C, c + 1) : 0;
    s.b = -1;
  }
  // entry of each worker's unit u1 - 1: scan the entries kThreads at a time
  int before = 0;
  for (int b0 = 0; b0 < l.count; b0 += kThreads) {
    const int b = b0 + tid;
    if (b0 > 0) {
      mine = Entry{};
      if (b < l.count) mine = entry_of<R, KT>(l, a, b, false);
      __syncthreads();  // the readers of scan are done
    }
    const int units = (direct ? mine.rt : mine.tiles) * a.Hkv;
    int incl = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int chunk = before;
    incl += before;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += scan[w];
      chunk += scan[w];
    }
    if (units > 0) {
#pragma unroll 1
      for (int w = 0; w < kWorkers; ++w) {
        const int last = shares[w].u1 - 1;
        if (incl - units <= last && last < incl) {
          shares[w].b = b;
          shares[w].off = last + 1 - (incl - units);
          shares[w].e = mine;
        }
      }
    }
    before = chunk;
    if (W <= before) break;  // uniform
  }
  __syncthreads();
}

// One list, all CTAs.
template <int R, int KT, int kThreads, int kWorkers>
__device__ __forceinline__ void make_shares(const PagedArgs& a, Share* shares) {
  __shared__ int red[3][kThreads / 32];
  __shared__ int scan[kThreads / 32];
  Entry mine;
  sum_entries<R, KT, kThreads>(a, a.list[0], mine, red);
  __syncthreads();
  share_list<R, KT, kThreads, kWorkers>(a, a.list[0], totals_of(red), mine,
                                                      blockIdx.x, gridDim.x, scan, shares);
}

// CTAs of `ctas` that work on list 1.  Costs are in key tiles of the few-row kernel, whose segments
// cost 8 more each (their queries to load and result to write; 23 sequences without keys of their
// own behind 24751: 35 us, 42 without the term), and a segment of the tensor-core kernel six of
// its key tiles (100 sequences of 700 keys behind three prefixes of 400: 59 us, 65 with three, 78
// without; 120 of 900 behind ten of 100: 52, 52 and 83).
__device__ __forceinline__ float list_cost(const PagedArgs& a, const KeyList& l, const Totals& t) {
  return l.mma ? (t.til + 6.f * t.seg) * a.mma_cost : t.til + 8.f * t.seg;
}
__device__ __forceinline__ int ctas_of_second(const PagedArgs& a, int ctas, const Totals (&t)[2]) {
  if (t[1].til == 0 || t[0].til == 0) return t[1].til == 0 ? 0 : ctas;
  const float c0 = list_cost(a, a.list[0], t[0]), c1 = list_cost(a, a.list[1], t[1]);
  return min(max(__float2int_rn(ctas * (c1 / (c0 + c1))), 1), ctas - 1);
}

// A worker's piece of one segment: key tiles [ta, te) of row tile r for key/value head hk.
struct Piece {
  int hk, r, ta, te;
  bool whole;  // no other worker has a part of the segment
  int unit;    // the segment's first unit
  int tiles;   // its key tiles
};

// Walks the pieces of a worker's share, last to first; e is the entry b of the current piece.
// Only the last unit's row tile is searched for: the ones before it follow by counting down.
template <int R, int KT>
struct Walk {
  int u0, u1;   // what is left of the share
  int b, hk, r; // the next piece's entry, key/value head and row tile (r < 0: the head before)
  int te;       // end of the first piece's key tiles; then -1: all of the row tile's
  bool direct;
  Entry e;

  __host__ __device__ Walk(const PagedArgs& a, const KeyList& l, const Share& sh)
      : u0(sh.u0), u1(sh.b < 0 ? sh.u0 : sh.u1), b(sh.b), hk(0), r(0), te(-1), direct(sh.direct),
        e(sh.e) {
    if (u0 >= u1) return;
    const int per_head = direct ? e.rt : e.tiles;
    hk = (sh.off - 1) / per_head;
    int rem = sh.off - 1 - hk * per_head;
    if (direct) {
      r = rem;
      return;
    }
    for (int n; rem >= (n = tiles_of<R, KT>(e, l.causal, a.G, r)); ++r) rem -= n;
    te = rem + 1;
  }
  __host__ __device__ bool next(const PagedArgs& a, const KeyList& l, Piece& p) {
    if (u0 >= u1) return false;
    if (r < 0) {
      if (--hk < 0) {
        do {                           // the entry before with tokens
          if (--b < 0) return false;   // cannot happen while u1 > u0
          e = entry_of<R, KT>(l, a, b, false);
        } while (e.rt == 0);
        hk = a.Hkv - 1;
      }
      r = e.rt - 1;
    }
    p.hk = hk;
    p.r = r--;
    p.tiles = tiles_of<R, KT>(e, l.causal, a.G, p.r);
    if (direct) {
      p.ta = 0;
      p.te = p.tiles;
      p.whole = true;
      p.unit = --u1;
      return true;
    }
    p.te = te >= 0 ? te : p.tiles;
    te = -1;
    p.unit = u1 - p.te;
    const int take = min(p.te, u1 - u0);
    p.ta = p.te - take;
    p.whole = take == p.tiles;
    u1 -= take;
    return true;
  }
};

// (first worker, number of workers) of the segment that this worker begins.
__host__ __device__ __forceinline__ int2 span_of(const Share& sh, const Piece& p) {
  const int last = p.whole ? sh.worker : share_owner(sh.W, sh.C, p.unit + p.tiles - 1);
  return make_int2(sh.worker, last - sh.worker + 1);
}

}  // namespace fa
