// Attention of a few query rows over a paged key/value cache: what a warp does.
//
// O = softmax(scale q K^T) V for the queries of one sequence that share a key/value head (group
// members x new tokens), 16 rows at a time: each K, V element is used by at most 16 rows, so the
// kernel is bound by reading the cache once.  Every warp is a worker of its own (paged_plan.cuh):
// it takes an equal share of all keys, copies 16 keys a step with cp.async into a private ring of
// shared-memory stages (keys past the length become zeros, whatever the page holds there),
// computes S (m16n8k16), the online softmax and O += P V from the ring, and writes its result or
// its part of one straight from registers.  No barrier after the start: warps never wait for each
// other, and a warp's ring goes on with the next piece while the last one is written.  (With 8
// warps on one segment and a merge in shared memory at each piece's end, 1024 segments of about
// 512 keys took 81 us instead of the copies' 40.)  mma.sync is enough here: one multiply-add a
// row for each 2-byte element is 16 flops a byte at 16 rows, 16 to 18% of the tensor pipe at the
// memory's rate (measured).
#pragma once

#include <type_traits>

#include "fa_internal.h"
#include "fa_paged.h"
#include "paged_plan.cuh"
#include "sm103.cuh"

namespace fa {

namespace rows16 {

constexpr int kWarps = kPagedWarps, kThreads = 32 * kWarps;
constexpr int R = kPagedRows;
constexpr int KT = kPagedKeys;        // keys of a step, and of a tile
constexpr float kLn2 = 0.693147180559945309f;

// One CTA per SM: 8 warps x stages of 16 keys (192 KB: with all but one stage of each in flight,
// 128 to 160 KB cover the latency of memory at full rate).
template <int D>
struct PagedLayout {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr uint32_t kHalf = KT * D * 2u;                // K or V of a step
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr uint32_t kBytes = kWarps * kStages * kStage;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;  // 0: the 16 bytes become zeros, src is not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte granule g of key row r in a step's K or V: granules are permuted within
// each 128 bytes by the row, so the eight rows of an ldmatrix fall into different banks.
template <int D>
__device__ __forceinline__ uint32_t step_offset(uint32_t r, uint32_t g) {
  return r * (D * 2u) + ((g ^ (r & 7u)) << 4);  // the xor stays within the granule's 128 bytes
}

// What a warp needs to copy the steps of a piece.
struct Source {
  const int32_t* trow;  // block-table row
  int hk, len;          // key/value head, keys
  int first, steps;     // key tile of step 0, number of steps
  int pages;            // lane i: page of step (issue & ~31) + i
  static constexpr KeyMode kMode = kAllKeys;
  struct Place {
    const int32_t* row;  // block-table row
    int key, len;        // first key of a step and the keys behind that row
    bool shared;         // of a prefix
  };
  __device__ Place place(int st) const { return {trow, (first + st) * KT, len, false}; }
};

// The same with the keys of a shared prefix in front (key tiles 0 .. pre - 1).
struct PrefixedSource : Source {
  const int32_t* prow;
  int pre, plen;
  __device__ Place place(int st) const {
    const int t = first + st;
    return t < pre ? Place{prow, t * KT, plen, true} : Place{trow, (t - pre) * KT, len, false};
  }
};

// Keys of which a tree hides some.
struct TreeSource : Source {
  static constexpr KeyMode kMode = kTreeKeys;
};

__device__ __forceinline__ Source source_of(const KeyList& l, const Walk<R, KT>& w,
                                            const Piece& p) {
  Source s;
  s.trow = l.table + static_cast<int64_t>(w.b) * l.max_pages;
  s.hk = p.hk;
  s.len = w.e.len;
  s.first = p.ta;
  s.steps = min(p.te, (w.e.len + KT - 1) / KT) - p.ta;  // none for an entry without keys
  s.pages = -1;
  return s;
}

// Copies step st into its stage (zeros for keys past the length and, reported, for a page outside
// the pool); every call commits a group, empty past the last step.
template <int D, typename Src>
__device__ __forceinline__ void issue_step(const PagedArgs& a, const KeyList& l, Src& s, int st,
                                           uint32_t ring, int lane) {
  using L = PagedLayout<D>;
  constexpr int S = L::kStages, GR = D / 8;  // granules of a row
  if (st < s.steps) {
    if ((st & 31) == 0) {
      const auto p = s.place(st + lane);
      const int max_pages = p.shared ? a.list[1].max_pages : l.max_pages;
      s.pages = st + lane < s.steps
                    ? resolve_page(p.row, max_pages, a.num_pages, a.page_shift, p.key)
                    : 0;
    }
    const int page = __shfl_sync(~0u, s.pages, st & 31);
    const auto p = s.place(st);
    const int slot = st % S;
    if (page < 0 && lane == 0) atomicCAS(a.status, 0, kErrIndex);
    const int64_t base = (((static_cast<int64_t>(max(page, 0)) * a.Hkv + s.hk) << a.page_shift) +
                          (p.key & ((1 << a.page_shift) - 1))) * D;
    const uint32_t dst = ring + slot * L::kStage;
#pragma unroll
    for (int i = 0; i < KT * GR / 32; ++i) {
      const int r = (i * 32 + lane) / GR, g = (i * 32 + lane) % GR;
      const bool valid = page >= 0 && p.key + r < p.len;
      const int64_t off = valid ? base + r * D + g * 8 : 0;
      cp_async16(dst + step_offset<D>(r, g), a.k_cache + off, valid);
      cp_async16(dst + L::kHalf + step_offset<D>(r, g), a.v_cache + off, valid);
    }
  }
  cp_commit();
}

// The keys of the pages selected for one token and key/value head, in the order of its list.
struct SelectedSource {
  const int32_t *trow, *list;  // block-table row of the token's sequence, its pages
  int hk, len;                 // key/value head, keys that the token sees
  int first, steps;
  int pages, keys;  // lane i: page (none: -1) and first key of step (issue & ~31) + i
  bool live;        // the token belongs to a sequence
  int* at;          // shared memory: first key of the step in each stage
  static constexpr KeyMode kMode = kSelectedKeys;
};
constexpr int kNoKey = 0x7fffff00;  // behind every key: lengths are at most this

// Entry of the list for step `st` of lane 0, + i of lane i (none: -1).
__device__ __forceinline__ int listed_page(const PagedArgs& a, const SelectedSource& s, int st, int steps, int lane) {
  return st + lane < steps ? __ldg(s.list + ((s.first + st + lane) >> (a.page_shift - 4))) : -1;
}
// Where that step's keys are: page `i` of the sequence, whose entry of the block table is `page`.  An
// entry of the list that names no page, or one behind what the token sees, has no keys.
__device__ __forceinline__ void locate(const PagedArgs& a, SelectedSource& s, int st, int i, int page, int lane) {
  s.pages = -1;
  s.keys = kNoKey;
  if (i >= 0 && i < (s.len + (1 << a.page_shift) - 1) >> a.page_shift) {
    s.keys = (i << a.page_shift) + ((s.first + st + lane) & ((1 << (a.page_shift - 4)) - 1)) * KT;
    if (page >= 0 && page < a.num_pages) s.pages = page;
    else atomicCAS(a.status, 0, kErrIndex);
  }
}
__device__ __forceinline__ int table_entry(const KeyList& l, const SelectedSource& s, int i) {
  return i >= 0 && i < l.max_pages ? __ldg(s.trow + i) : -1;
}

// The first steps' pages are looked up on the way: the list while the token's sequence is searched
// for, the block table together with its length.
__device__ __forceinline__ SelectedSource selected_source(const PagedArgs& a, const KeyList& l,
                                                          const Walk<R, KT>& w, const Piece& p,
                                                          int* at, int lane) {
  SelectedSource s;
  s.hk = p.hk;
  s.first = p.ta;
  s.at = at;
  const int t = w.e.start, most = max(min(p.te, (l.max_len + KT - 1) / KT) - p.ta, 0);
  s.list = a.pages + (static_cast<int64_t>(t) * a.Hkv + p.hk) * a.top;
  const int i = listed_page(a, s, 0, most, lane);
  const int b = token_sequence_group<32>(a.seq_cu, a.seqs, t, lane, ~0u);
  s.trow = l.table + static_cast<int64_t>(max(b, 0)) * l.max_pages;
  const int page = table_entry(l, s, i);
  int start = 0, n = 0;
  if (b >= 0) token_bounds(a.seq_cu, b, a.total, start, n);
  s.live = b >= 0 && t >= start && t < start + n;
  if (b >= 0 && !s.live && lane == 0) atomicCAS(a.status, 0, kErrIndex);  // do not ascend
  const int64_t reach = static_cast<int64_t>(l.max_pages) << a.page_shift;
  const int given = s.live ? __ldg(a.seq_lens + b) : 0;
  const int len = min(max(given, 0), static_cast<int>(min(reach, static_cast<int64_t>(kNoKey))));
  if (given != len && lane == 0) atomicCAS(a.status, 0, kErrIndex);
  s.len = min(max(len - n + (t - start) + 1, 0), len);
  s.steps = s.len > 0 ? most : 0;
  locate(a, s, 0, i, page, lane);
  return s;
}

// issue_step for selected pages.
template <int D>
__device__ __forceinline__ void issue_step(const PagedArgs& a, const KeyList& l, SelectedSource& s,
                                           int st, uint32_t ring, int lane) {
  using L = PagedLayout<D>;
  constexpr int S = L::kStages, GR = D / 8;
  if (st < s.steps) {
    if ((st & 31) == 0 && st > 0) {
      const int i = listed_page(a, s, st, s.steps, lane);
      locate(a, s, st, i, table_entry(l, s, i), lane);
    }
    const int page = __shfl_sync(~0u, s.pages, st & 31), key = __shfl_sync(~0u, s.keys, st & 31);
    const int slot = st % S;
    if (lane == 0) s.at[slot] = key;
    const int64_t base = (((static_cast<int64_t>(max(page, 0)) * a.Hkv + s.hk) << a.page_shift) +
                          (key & ((1 << a.page_shift) - 1))) * D;
    const uint32_t dst = ring + slot * L::kStage;
#pragma unroll
    for (int i = 0; i < KT * GR / 32; ++i) {
      const int r = (i * 32 + lane) / GR, g = (i * 32 + lane) % GR;
      const bool valid = page >= 0 && key + r < s.len;
      const int64_t off = valid ? base + r * D + g * 8 : 0;
      cp_async16(dst + step_offset<D>(r, g), a.k_cache + off, valid);
      cp_async16(dst + L::kHalf + step_offset<D>(r, g), a.v_cache + off, valid);
    }
  }
  cp_commit();
}

// A row tile's queries as A fragments: the thread holds rows lane / 4 and lane / 4 + 8.
template <int D>
struct QRows {
  uint32_t qf[D / 16][4];
  int lim[2];   // keys below it are visible to the row
  int at[2];    // (token, head) of the row
  int head[2];
  int rows, lim_min;  // rows of the tile; the first row's limit, the smallest
  const uint32_t* tree[2];  // kTreeKeys: mask rows; the context ends at lim_min
};
template <int D, KeyMode M>
__device__ __forceinline__ QRows<D> load_rows(const PagedArgs& a, const KeyList& l, const Entry& e,
                                              const Piece& p, int lane) {
  QRows<D> x;
  const int row0 = p.r * R, rows = min(R, e.nc * a.G - row0);
  x.rows = rows;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int rr = (lane >> 2) + 8 * i, tok = (row0 + rr) / a.G;
    x.lim[i] = rr < rows ? row_limit(e, l.causal, a.G, row0 + rr) : e.len;
    x.head[i] = p.hk * a.G + (row0 + rr - tok * a.G);
    x.at[i] = (e.start + tok) * a.H + x.head[i];
    if constexpr (M == kTreeKeys)
      x.tree[i] = a.tree + static_cast<int64_t>(e.start + (rr < rows ? tok : 0)) * a.tree_words;
    const __nv_bfloat16* qp = a.q + static_cast<int64_t>(x.at[i]) * D + (lane & 3) * 2;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      x.qf[k][i] = rr < rows ? *reinterpret_cast<const uint32_t*>(qp + k * 16) : 0u;
      x.qf[k][i + 2] = rr < rows ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + 8) : 0u;
    }
  }
  x.lim_min = M == kTreeKeys ? e.len - e.n : row_limit(e, l.causal, a.G, row0);
  return x;
}

// Running O, maximum (log2 units) and sum of the thread's two rows.
template <int D>
struct Acc {
  float o[D / 8][4], m[2], sum[2];
  __device__ Acc() : m{-INFINITY, -INFINITY}, sum{0.f, 0.f} {
#pragma unroll
    for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  }
};

// The keys of a source, whose first S - 1 steps have been issued.
template <int D, typename Src>
__device__ __forceinline__ void scan_keys(const PagedArgs& a, const KeyList& l, Src& src,
                                          const QRows<D>& x, uint32_t ring, int lane, Acc<D>& c) {
  using L = PagedLayout<D>;
  constexpr int S = L::kStages;
  for (int st = 0; st < src.steps; ++st) {
    cp_wait<S - 2>();
    __syncwarp();
    const uint32_t kb = ring + (st % S) * L::kStage, vb = kb + L::kHalf;
    // S = Q K^T: 16 rows x 16 keys
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    {
      const uint32_t r = (lane & 7) + ((lane >> 4) << 3), gh = (lane >> 3) & 1;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t f[4];
        ldsm4(kb + step_offset<D>(r, 2 * k + gh), f);
        mma16816(s[0], x.qf[k], f[0], f[1]);
        mma16816(s[1], x.qf[k], f[2], f[3]);
      }
    }
    if constexpr (Src::kMode == kAllKeys) {
      const auto p = src.place(st);
      if (p.key + KT > (p.shared ? p.len : x.lim_min)) {  // all of a prefix is visible
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = p.key + n * 8 + (lane & 3) * 2 + (k & 1);
            if (key >= (p.shared ? p.len : x.lim[k >> 1])) s[n][k] = -INFINITY;
          }
      }
    } else {
      int key0;
      uint32_t see[2];  // bit i: the row sees key key0 + i
      bool all;
      if constexpr (Src::kMode == kSelectedKeys) {
        key0 = src.at[st % S];
        all = key0 + KT <= src.len;
        see[0] = see[1] = (1u << min(max(src.len - key0, 0), KT)) - 1u;
      } else {
        key0 = src.place(st).key;
        all = key0 + KT <= x.lim_min;
        if (!all) {
          const uint32_t there = (1u << min(max(src.len - key0, 0), KT)) - 1u;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            see[i] = tree_window(x.tree[i], a.tree_words, key0 - x.lim_min) & there;
        }
      }
      if (!all) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (!((see[k >> 1] >> (n * 8 + (lane & 3) * 2 + (k & 1))) & 1u)) s[n][k] = -INFINITY;
      }
    }
    // online softmax; the row maximum is shared by the four lanes of a row, the sum is
    // joined at the end
    bool moved = false;
    float alpha[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx =
          fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2)) * a.scale_log2;
      alpha[i] = 1.f;
      if (mx > c.m[i]) {
        alpha[i] = ex2(c.m[i] - mx);
        c.m[i] = mx;
        moved = true;
      }
      const float ref = c.m[i] == -INFINITY ? 0.f : c.m[i];
      float total = 0.f;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // the scale is never 0, so a hidden score stays -inf and weighs 0
          const float e = ex2(fmaf(s[n][2 * i + k], a.scale_log2, -ref));
          s[n][2 * i + k] = e;
          total += e;
        }
      c.sum[i] = c.sum[i] * alpha[i] + total;
    }
    if (__any_sync(~0u, moved)) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        c.o[n][0] *= alpha[0];
        c.o[n][1] *= alpha[0];
        c.o[n][2] *= alpha[1];
        c.o[n][3] *= alpha[1];
      }
    }
    // O += P V; P rounded to bf16 (half a step, 2^-8, as in fa_fwd), its sum is not
    const uint32_t pf[4] = {pack_bf16(s[0][0], s[0][1]), pack_bf16(s[0][2], s[0][3]),
                            pack_bf16(s[1][0], s[1][1]), pack_bf16(s[1][2], s[1][3])};
    {
      const uint32_t r = lane & 15, gh = lane >> 4;
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        uint32_t f[4];
        ldsm4_t(vb + step_offset<D>(r, 2 * n + gh), f);
        mma16816(c.o[2 * n], pf, f[0], f[1]);
        mma16816(c.o[2 * n + 1], pf, f[2], f[3]);
      }
    }
    __syncwarp();  // every lane has read stage st % S before it is filled again
    issue_step<D>(a, l, src, st + S - 1, ring, lane);
  }
}

// The keys of a piece; `at`: a shared-memory word for each stage of the ring (selected pages).
template <KeyMode M>
__device__ __forceinline__ auto make_source(const PagedArgs& a, const KeyList& l,
                                            const Walk<R, KT>& w, const Piece& p, int* at, int lane) {
  if constexpr (M == kSelectedKeys) {
    return selected_source(a, l, w, p, at, lane);
  } else if constexpr (M == kTreeKeys) {
    return TreeSource{source_of(l, w, p)};
  } else {
    return source_of(l, w, p);
  }
}
template <typename Src>
__device__ __forceinline__ bool has_result(const Src& s) {
  if constexpr (Src::kMode == kSelectedKeys) return s.live;
  return true;
}

// A worker's share of a list's keys (one warp).
template <int D, KeyMode M>
__device__ __forceinline__ void work(const PagedArgs& a, const KeyList& l,
                                     const PartialLayout& part, float* rowbuf, const Share& sh,
                                     uint32_t ring, int* at, int lane) {
  using L = PagedLayout<D>;
  constexpr int S = L::kStages;
  if (sh.u0 >= sh.u1 || sh.b < 0) return;
  Walk<R, KT> walk(a, l, sh);
  Piece next_piece;
  bool more = walk.next(a, l, next_piece);
  auto src = make_source<M>(a, l, walk, next_piece, at, lane);
  for (int st = 0; st < S - 1; ++st) issue_step<D>(a, l, src, st, ring, lane);
  while (more) {
    const Piece piece = next_piece;
    const Entry e = walk.e;
    const int tile = row_tile0(e.start, a.G, R, walk.b) + piece.r;
    if (lane == 0 && piece.ta == 0)  // this worker begins the segment
      part.spans[static_cast<int64_t>(piece.hk) * part.span_tiles + tile] = span_of(sh, piece);

    const QRows<D> x = load_rows<D, M>(a, l, e, piece, lane);
    Acc<D> c;
    scan_keys<D>(a, l, src, x, ring, lane, c);
    const bool result = has_result(src);
    // every stage has been read: the next piece's copies start here
    more = walk.next(a, l, next_piece);
    if (more) {
      src = make_source<M>(a, l, walk, next_piece, at, lane);
      for (int st = 0; st < S - 1; ++st) issue_step<D>(a, l, src, st, ring, lane);
    }

    // ---- the rows' results, or this worker's part of them
    const bool final_out = piece.whole && rowbuf == nullptr;
    float* slot = part.slots + (static_cast<int64_t>(sh.worker) * 2 + (piece.ta == 0)) *
                                     (R * (D + 2));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c.sum[i] += __shfl_xor_sync(~0u, c.sum[i], 1);
      c.sum[i] += __shfl_xor_sync(~0u, c.sum[i], 2);
      const int rr = (lane >> 2) + 8 * i;
      if (rr >= x.rows || !result) continue;
      const float inv = c.sum[i] > 0.f ? 1.f / c.sum[i] : (c.sum[i] == 0.f ? 0.f : c.sum[i]);  // NaN stays
      if (final_out) {
        uint32_t* dst =
            reinterpret_cast<uint32_t*>(a.o + static_cast<int64_t>(x.at[i]) * D) + (lane & 3);
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          dst[n * 4] = pack_bf16(c.o[n][2 * i] * inv, c.o[n][2 * i + 1] * inv);
      } else {
        float* row = piece.whole ? rowbuf + static_cast<int64_t>(x.at[i]) * D : slot + rr * D;
        float2* dst = reinterpret_cast<float2*>(row) + (lane & 3);
#pragma unroll
        for (int n = 0; n < D / 8; ++n) dst[n * 4] = make_float2(c.o[n][2 * i], c.o[n][2 * i + 1]);
      }
      if ((lane & 3) == 0) {
        if (final_out) {
          const int t = (x.at[i] - x.head[i]) / a.H;
          a.lse[static_cast<int64_t>(x.head[i]) * a.total + t] =
              c.sum[i] == 0.f ? -INFINITY : (c.m[i] + log2f(c.sum[i])) * kLn2;
        } else {
          float* st = piece.whole ? rowbuf + static_cast<int64_t>(a.total) * a.H * D + x.at[i]
                                  : slot + R * D + rr;
          st[0] = c.m[i];
          st[piece.whole ? a.total * a.H : R] = c.sum[i];
        }
      }
    }
  }
  cp_wait<0>();
}

// Few segments: the 8 warps of a CTA take an eighth of a piece's keys each and meet in shared memory
// (their own rings, whose copies have all been read), so that short segments leave nothing to join
// and long ones an eighth of the parts.  The Share is the CTA's.  kPrefix: a sequence's keys are those
// of its group's prefix and then its own; the prefix is read once per sequence, from L2.
template <int D, bool kPrefix, KeyMode M>
__device__ __forceinline__ void work_together(const PagedArgs& a, const KeyList& l,
                                              const PartialLayout& parts, const Share& sh,
                                              uint8_t* smem, int* at, int warp, int lane) {
  static_assert(!kPrefix || M == kAllKeys, "prefixes have all of their keys");
  using L = PagedLayout<D>;
  constexpr int S = L::kStages, P = D + 8;  // row pitch of a warp's O in floats
  constexpr uint32_t kRing = S * L::kStage;
  static_assert((R * P + 2 * R) * 4 <= kRing, "a warp's O, maxima and sums fit its ring");
  const uint32_t ring = smem_u32(smem) + warp * kRing;
  Walk<R, KT> walk(a, l, sh);
  Piece piece;
  while (walk.next(a, l, piece)) {
    const Entry& e = walk.e;
    Piece own = piece;
    if constexpr (M == kSelectedKeys) {  // looked up for the warp's own steps
      const int64_t n = piece.te - piece.ta;
      own.te = piece.ta + static_cast<int>((warp + 1) * n / kWarps);
      own.ta = piece.ta + static_cast<int>(warp * n / kWarps);
    }
    auto source = make_source<M>(a, l, walk, own, at, lane);
    std::conditional_t<kPrefix, PrefixedSource, decltype(source)> src;
    static_cast<decltype(source)&>(src) = source;
    if constexpr (kPrefix) {
      const KeyList& pl = a.list[1];
      const int g = token_sequence_group<32>(pl.group_cu, pl.count, walk.b, lane, ~0u);
      // a sequence of no group has no prefix
      src.plen = g >= 0 ? entry_of<R, KT>(pl, a, g, false).len : 0;
      src.prow = pl.table + static_cast<int64_t>(max(g, 0)) * pl.max_pages;
      src.pre = (src.plen + KT - 1) / KT;
      src.steps += src.pre;
    }
    if (threadIdx.x == 0 && piece.ta == 0)  // this CTA begins the segment
      parts.spans[static_cast<int64_t>(piece.hk) * parts.span_tiles +
                  row_tile0(e.start, a.G, R, walk.b) + piece.r] = span_of(sh, piece);
    if constexpr (M != kSelectedKeys) {
      const int t0 = static_cast<int>(static_cast<int64_t>(warp) * src.steps / kWarps);
      const int t1 = static_cast<int>(static_cast<int64_t>(warp + 1) * src.steps / kWarps);
      src.first += t0;
      src.steps = t1 - t0;
    }
    for (int st = 0; st < S - 1; ++st) issue_step<D>(a, l, src, st, ring, lane);
    const QRows<D> x = load_rows<D, M>(a, l, e, piece, lane);
    Acc<D> c;
    scan_keys<D>(a, l, src, x, ring, lane, c);
    const bool result = has_result(src);
    float* mine = reinterpret_cast<float*>(smem + warp * kRing);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c.sum[i] += __shfl_xor_sync(~0u, c.sum[i], 1);
      c.sum[i] += __shfl_xor_sync(~0u, c.sum[i], 2);
      const int rr = (lane >> 2) + 8 * i;
      float2* dst = reinterpret_cast<float2*>(mine + rr * P) + (lane & 3);
#pragma unroll
      for (int n = 0; n < D / 8; ++n) dst[n * 4] = make_float2(c.o[n][2 * i], c.o[n][2 * i + 1]);
      if ((lane & 3) == 0) {
        mine[R * P + rr] = c.m[i];
        mine[R * P + R + rr] = c.sum[i];
      }
    }
    __syncthreads();
    // 16 threads a row, E elements each, over the warps in the order of their keys
    constexpr int E = D / 16;
    const int rr = threadIdx.x / 16, part = threadIdx.x % 16;
    float m[kWarps], s[kWarps], top = -INFINITY, sum = 0.f, o[E];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* from = reinterpret_cast<const float*>(smem + w * kRing) + R * P + rr;
      m[w] = from[0];
      s[w] = from[R];
      top = fmaxf(top, m[w]);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      // no visible key: weight 0 (NaN stays)
      const float f = m[w] == -INFINITY ? (s[w] == 0.f ? 0.f : s[w]) : ex2(m[w] - top);
      sum = fmaf(f, s[w], sum);
      const float4* from = reinterpret_cast<const float4*>(
          reinterpret_cast<const float*>(smem + w * kRing) + rr * P + part * E);
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const float4 v = from[i];
        o[4 * i] = fmaf(f, v.x, o[4 * i]);
        o[4 * i + 1] = fmaf(f, v.y, o[4 * i + 1]);
        o[4 * i + 2] = fmaf(f, v.z, o[4 * i + 2]);
        o[4 * i + 3] = fmaf(f, v.w, o[4 * i + 3]);
      }
    }
    if (!result) {
    } else if (rr < x.rows && !piece.whole) {
      float* slot = parts.slots + (static_cast<int64_t>(sh.worker) * 2 + (piece.ta == 0)) *
                                      (R * (D + 2));
      float4* dst = reinterpret_cast<float4*>(slot + rr * D + part * E);
#pragma unroll
      for (int i = 0; i < E / 4; ++i)
        dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      if (part == 0) {
        slot[R * D + rr] = top;
        slot[R * D + R + rr] = sum;
      }
    } else if (rr < x.rows) {
      const int row = piece.r * R + rr, tok = row / a.G;
      const int head = piece.hk * a.G + (row - tok * a.G);
      const int64_t at = static_cast<int64_t>(e.start + tok) * a.H + head;
      const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
      uint2* dst = reinterpret_cast<uint2*>(a.o + at * D + part * E);
#pragma unroll
      for (int i = 0; i < E / 4; ++i)
        dst[i] = make_uint2(pack_bf16(o[4 * i] * inv, o[4 * i + 1] * inv),
                            pack_bf16(o[4 * i + 2] * inv, o[4 * i + 3] * inv));
      if (part == 0)
        a.lse[static_cast<int64_t>(head) * a.total + e.start + tok] =
            sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
    __syncthreads();  // the rings are free for the next segment
  }
  cp_wait<0>();
}

}  // namespace rows16

}  // namespace fa
