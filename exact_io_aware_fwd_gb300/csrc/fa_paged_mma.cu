// Attention of many query rows over a paged key/value cache on the tcgen05 tensor cores: chunks
// of prompts, and all the queries of a batch against the prefix that they share.
//
// The method is fa_fwd's (two 128-row query tiles per CTA that alternate on the tensor core, one
// thread per row in the softmax, O~ rescaled in tensor memory only when a row's maximum moved);
// what differs is where rows and keys come from and where results go:
//  * a row tile is 256 consecutive (token, group member) rows of one key/value head, so the heads
//    of a group share every K, V tile; rows are gathered with plain loads into the swizzled Q
//    tiles (any group size), K and V come page by page through a TMA map of the pool, whose
//    out-of-range coordinate gives zeros for pages past the end or outside the pool;
//  * the rows of the last page past the sequence's end may hold anything (an infinity times a
//    zero weight would be NaN), so the softmax warps clear them in the V tile before P V;
//  * CTAs are persistent and take equal shares of all key tiles (paged_plan.cuh).  Warp 2 works
//    out the CTA's pieces and hands them to the other roles through a ring in shared memory, so
//    the TMA warp runs ahead into the next piece while the softmax warps finish the last one; a
//    segment that several CTAs share leaves float32 parts for the join kernel.
// A call with shared prefixes runs as one launch: the SMs are divided between the groups' prefixes
// and the sequences' own keys by what their key tiles cost (paged_plan.cuh, kLists == 2).
// A K or V element takes part in one multiply-add a row: 256 flops a byte at 256 rows, next to the
// balance of the measured peaks (280).  So one row tile is bound by the copies from memory, several
// row tiles a head, which share K and V in L2 (the chunk case reads each key once from memory), by
// the MMAs next to the softmax.
#include "fa_internal.h"
#include "fa_paged.h"
#include "paged_plan.cuh"
#include "paged_rows.cuh"
#include "sm103.cuh"

namespace fa {

namespace {

constexpr int kThreads = 384;  // warp 0: TMA, 1: MMA, 2: pieces, 4-7 and 8-11: softmax
constexpr int R = kPagedMmaRows;
constexpr int KT = kPagedMmaKeys;
constexpr float kLn2 = 0.693147180559945309f;

// What the roles need to know of a piece, in a ring of shared memory.
struct PieceInfo {
  int n[2];        // key tiles of each query tile: the first n of the piece's (kTwin: every other
                   // one); -1: no more pieces
  int ta;          // first key tile
  int hk, row0;    // key/value head, first row of the row tile
  int start, rows; // the entry's first token and its rows (computed tokens x group)
  int len, shift;  // keys, and keys minus tokens (row r sees shift + r / G + 1 keys if causal)
  int tile;        // row tile's index in the spans
  int whole;       // no other CTA works on the segment
  const int32_t* table;  // the entry's block-table row
};
constexpr int kRing = 4;
// Key tiles (positions) of the piece.
template <bool kTwin>
__device__ __forceinline__ int positions(int n0, int n1) {
  return kTwin ? n0 + n1 : max(n0, n1);
}

template <int D>
struct MmaLayout {
  static constexpr uint32_t kTile = 128u * D * 2u;
  static constexpr int kStages = D == 64 ? 4 : 2;
  // K and V in front of Q: 3% faster than the other way round (231 -> 223 us for 2 x 512 tokens over
  // 16384 keys).  192 KB and what is static fit the SM's 196 KB setting; a few KB more, such as a
  // gap between the buffers, take the next one, leave less L1 and cost 3%.
  static constexpr uint32_t kK = 0;
  static constexpr uint32_t kV = kK + kStages * kTile;
  static constexpr uint32_t kQ = kV + kStages * kTile;
  static constexpr uint32_t kBytes = kQ + 2 * kTile;
  static constexpr uint32_t kColS0 = 0, kColO0 = 256;
  static constexpr uint32_t kTmemCols = 512;
};

// Shared memory of a CTA: the tiles, or with two lists the rings of a CTA of few rows.
template <int D, int kLists>
__host__ __device__ constexpr uint32_t smem_of() {
  return kLists == 1 || MmaLayout<D>::kBytes > rows16::PagedLayout<D>::kBytes
             ? MmaLayout<D>::kBytes
             : rows16::PagedLayout<D>::kBytes;
}

// 32 bytes, 32-byte aligned.
__device__ __forceinline__ void st_v8(float* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// Key tiles of query tile t (rows [256 r + 128 t, + 128)) inside the piece's range.
__device__ __forceinline__ int tiles_in_piece(const Entry& e, const Piece& p, int causal, int G,
                                              int t) {
  const int r0 = p.r * R + 128 * t, rows = e.nc * G;
  if (r0 >= rows) return 0;
  const int lim = max(0, row_limit(e, causal, G, min(rows, r0 + 128) - 1));
  return max(0, min(p.te, (lim + KT - 1) / KT) - p.ta);
}

// kLists == 2: a call with shared prefixes, each list on its own part of the SMs.  The CTAs of a
// list of few rows do what paged_kernel does, with the softmax warps as the workers.
// kTwin: no entry has more than 128 rows, one query tile.  Both tile slots work on it, at alternate
// positions, and their results are joined at a piece's end: with one slot, the chain S, softmax,
// P V of a position is all that runs (126 sequences of 18 rows and 1576 keys 149 us, with one slot
// 166; d = 64, 16 of 36 rows and 8192 keys 67 and 82).  Here K runs a position ahead of V: a V
// stage is free only two positions later (211 us with K and V together).
// M: kAllKeys, or kTreeKeys (one list).
// A warp's results leave for the workspace 32 bytes a thread at a time, whole sectors (32 trees of 48 to 64
// tokens over 2048 to 8192 keys: 165.6 us, 168.4 with 16).  Of a tree, the queries of the next pieces are
// fetched into L2 (167.8; both: 164.2).  With two lists that is slower (128 sequences behind two prefixes of
// 32768 keys 137.5 us, without 136.0).
template <int D, int kLists, bool kTwin, KeyMode M>
__global__ void __launch_bounds__(kThreads, 1)
    paged_mma_kernel(const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedArgs a,
                     const uint64_t timeout_ns, const uint32_t smem_bytes) {
  using L = MmaLayout<D>;
  constexpr int S = L::kStages, P = D / 64;  // 64-column panels of a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  uint8_t* sm = smem_raw + pad;
  // what the roles signal through: static, so that its addresses are constants and take no registers
  __shared__ uint64_t q_full[1], k_full[S], k_empty[S], v_full[S], v_empty[S];
  __shared__ uint64_t s_full[2], p_full[2], o_full[2], mma_done[1], twin_full[1];
  __shared__ float twin_m[kTwin ? 128 : 1], twin_l[kTwin ? 128 : 1];
  __shared__ uint64_t piece_full[kRing], piece_empty[kRing];
  __shared__ PieceInfo pieces[kRing];
  __shared__ uint32_t tmem_slot[1];
  __shared__ volatile int abort_flag[1];
  __shared__ Share shares[kLists == 2 ? kPagedWarps : 1];
  const Ctl ctl{abort_flag, a.status, timeout_ns};
  const uint32_t warp = warp_id(), lane = lane_id();
  if (pad + smem_of<D, kLists>() > smem_bytes) {  // cannot happen: the array is aligned; never proceed
    if (threadIdx.x == 0) atomicCAS(a.status, 0, kErrLayout);
    return;
  }
  // nothing here depends on what earlier launches write
  if (warp == 0 && lane == 0) {
    *abort_flag = 0;
    mbar_init(q_full, 8);
    for (int s = 0; s < S; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_full[t], 1);
    }
    mbar_init(mma_done, 1);
    mbar_init(twin_full, 4);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], 10);  // TMA warp, MMA thread, 8 softmax warps
    }
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // the share of the list that this CTA works on
  touch(a);
  begin_launch();
  int li = 0;
  if constexpr (kLists == 1) {
    make_shares<R, KT, kThreads, 1>(a, shares);
  } else {
    __shared__ int red[2][3][kThreads / 32], scan[kThreads / 32];
    Entry mine[2];
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      Entry e;
      if (a.list[i].mma) sum_entries<R, KT, kThreads>(a, a.list[i], e, red[i]);
      else sum_entries<rows16::R, rows16::KT, kThreads>(a, a.list[i], e, red[i]);
      if (i == 0) mine[0] = e;
      else mine[1] = e;
    }
    __syncthreads();
    const Totals t[2] = {totals_of(red[0]), totals_of(red[1])};
    const int n1 = ctas_of_second(a, gridDim.x, t);
    li = static_cast<int>(blockIdx.x) < n1 ? 1 : 0;
    const int cta = li ? blockIdx.x : blockIdx.x - n1, ctas = li ? n1 : gridDim.x - n1;
    const Totals ti = li ? t[1] : t[0];
    const Entry own = li ? mine[1] : mine[0];
    if (a.list[li].mma)
      share_list<R, KT, kThreads, 1>(a, a.list[li], ti, own, cta, ctas, scan, shares);
    else
      share_list<rows16::R, rows16::KT, kThreads, kPagedWarps>(
          a, a.list[li], ti, own, cta, ctas, scan, shares);
  }
  const KeyList& l = a.list[li];
  const PartialLayout& part = a.part[li];
  float* const rowbuf = a.rowbuf[li];
  const bool few_rows = kLists == 2 && !l.mma;
  const Share& sh = shares[0];
  const uint32_t tmem = *tmem_slot;
  const uint32_t sbase = smem_u32(sm);
  // Registers: the launch gives 384 x 168; warps 0-3 keep 56 and the softmax warps take 224
  // (128 x 56 + 256 x 224 = 384 x 168), enough for a row's scores and weights: with 168 for all,
  // or 72 / 216, the spills in the loop cost up to 15% (2 x 512 tokens over 16384 keys).
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (few_rows) {
    } else if (warp == 2) {
      // ================= the CTA's pieces; of a tree, with their queries on the way to L2
      constexpr bool kFetch = M == kTreeKeys;
      if (kFetch || lane == 0) {
        Walk<R, KT> walk(a, l, sh);
        const Entry& e = walk.e;
        Piece piece;
        for (int i = 0;; ++i) {
          const bool more = walk.next(a, l, piece);
          const uint32_t parity = ((i / kRing) & 1) ^ 1;
          if (!(kFetch ? mbar_wait_warp(&piece_empty[i % kRing], parity, ctl)
                       : mbar_wait(&piece_empty[i % kRing], parity, ctl)))
            break;
          if (lane == 0) {
            PieceInfo& p = pieces[i % kRing];
            if (more) {
              const int n0 = tiles_in_piece(e, piece, l.causal, a.G, 0);
              p.n[0] = kTwin ? (n0 + 1) / 2 : n0;
              p.n[1] = kTwin ? n0 / 2 : tiles_in_piece(e, piece, l.causal, a.G, 1);
              p.ta = piece.ta;
              p.hk = piece.hk;
              p.row0 = piece.r * R;
              p.start = e.start;
              p.rows = e.nc * a.G;
              p.len = e.len;
              p.shift = e.len - e.n;
              p.tile = row_tile0(e.start, a.G, R, walk.b) + piece.r;
              p.whole = piece.whole;
              p.table = l.table + static_cast<int64_t>(walk.b) * l.max_pages;
              if (piece.ta == 0)  // this CTA begins the segment
                part.spans[static_cast<int64_t>(piece.hk) * part.span_tiles + p.tile] =
                    span_of(sh, piece);
            } else {
              p.n[0] = p.n[1] = -1;
            }
            mbar_arrive(&piece_full[i % kRing]);
          }
          if (!more) break;
          if constexpr (!kFetch) continue;
          // rows of one token and key/value head are neighbours
          const int rows = min(e.nc * a.G - piece.r * R, R), line = D * 2 / 128;
          for (int x = lane; x < rows * line; x += 32) {
            const int gr = piece.r * R + x / line, tok = gr / a.G;
            const char* q = reinterpret_cast<const char*>(
                a.q + (static_cast<int64_t>(e.start + tok) * a.H + piece.hk * a.G + (gr - tok * a.G)) * D);
            prefetch_l2(q + x % line * 128);
          }
        }
      }
    } else if (warp == 0) {
      // ================= TMA producer: one box (page x 64 columns) per lane
      const int page_size = 1 << a.page_shift, pages = KT >> a.page_shift;
      const int pg = lane & (pages - 1), panel = lane / pages;
      const bool mine = panel < P;
      int jk = 0, jv = 0;  // positions whose K and V copies have been issued
      bool ok = true;
      for (int i = 0;; ++i) {
        if (!(ok = mbar_wait_warp(&piece_full[i % kRing], (i / kRing) & 1, ctl))) break;
        const PieceInfo& p = pieces[i % kRing];
        const int npos = positions<kTwin>(p.n[0], p.n[1]);
        const int32_t* trow = p.table;
        const int len = p.len, hk = p.hk, ta = p.ta;
        __syncwarp();
        if (lane == 0) mbar_arrive(&piece_empty[i % kRing]);  // all of it is in registers
        if (npos < 0) break;
        // page of this lane's box at key tile kt: the map's out-of-range coordinate, which reads
        // as zeros, past the end and (reported) for a page outside the pool
        auto find = [&](int kt) {
          const int key = kt * KT + pg * page_size;
          if (key >= len) return a.num_pages * a.Hkv;
          const int page = resolve_page(trow, l.max_pages, a.num_pages, a.page_shift, key);
          if (page < 0) atomicCAS(a.status, 0, kErrIndex);
          return page < 0 ? a.num_pages * a.Hkv : page * a.Hkv + hk;
        };
        if constexpr (kTwin) {
          // K runs one position ahead of V: a V stage is free only after its P V
          int zk = npos > 0 ? find(ta) : 0, zv = zk;  // K's and V's pages of the next copies
          for (int j = 0; j <= npos && npos > 0; ++j) {
            if (j < npos) {
              const int s = jk % S;
              if (!(ok = mbar_wait_warp(&k_empty[s], ((jk / S) & 1) ^ 1, ctl))) break;
              if (lane == 0) mbar_arrive_expect_tx(&k_full[s], L::kTile);
              __syncwarp();
              const uint32_t at = s * L::kTile + panel * 16384 + pg * (page_size * 128);
              if (mine) tma_load_3d(sm + L::kK + at, &tmK, &k_full[s], panel * 64, 0, zk);
              ++jk;
            }
            if (j > 0) {
              const int s = jv % S;
              if (!(ok = mbar_wait_warp(&v_empty[s], ((jv / S) & 1) ^ 1, ctl))) break;
              if (lane == 0) mbar_arrive_expect_tx(&v_full[s], L::kTile);
              __syncwarp();
              const uint32_t at = s * L::kTile + panel * 16384 + pg * (page_size * 128);
              if (mine) tma_load_3d(sm + L::kV + at, &tmV, &v_full[s], panel * 64, 0, zv);
              ++jv;
            }
            zv = zk;
            if (j + 1 < npos) zk = find(ta + j + 1);
          }
        } else {
          int z = 0, z_next = npos > 0 ? find(ta) : 0;
          for (int j = 0; j < npos; ++j) {
            const int s = jk % S;
            const uint32_t ph = (jk / S) & 1;
            z = z_next;
            if (j + 1 < npos) z_next = find(ta + j + 1);
            if (!(ok = mbar_wait_warp(&k_empty[s], ph ^ 1, ctl))) break;
            if (lane == 0) mbar_arrive_expect_tx(&k_full[s], L::kTile);
            __syncwarp();
            const uint32_t at = s * L::kTile + panel * 16384 + pg * (page_size * 128);
            if (mine) tma_load_3d(sm + L::kK + at, &tmK, &k_full[s], panel * 64, 0, z);
            ++jk;
            if (!(ok = mbar_wait_warp(&v_empty[s], ph ^ 1, ctl))) break;
            if (lane == 0) mbar_arrive_expect_tx(&v_full[s], L::kTile);
            __syncwarp();
            if (mine) tma_load_3d(sm + L::kV + at, &tmV, &v_full[s], panel * 64, 0, z);
            ++jv;
          }
        }
        if (!ok) break;
      }
      // no copy into this CTA's shared memory may still be in flight when the CTA exits
      if (lane == 0) {
        for (int j = max(0, jk - S); j < jk; ++j) drain_wait(&k_full[j % S], (j / S) & 1, ctl);
        for (int j = max(0, jv - S); j < jv; ++j) drain_wait(&v_full[j % S], (j / S) & 1, ctl);
      }
    } else if (warp == 1) {
      // ================= MMA issuer
      if (lane == 0) {
        constexpr uint32_t idS = idesc_bf16(128, 128, false, false);  // S = Q K^T, both K-major
        constexpr uint32_t idO = idesc_bf16(128, D, false, true);     // O += P V, V is MN-major
        int base = 0, segs = 0;  // positions and pieces before this one
        int issued[2] = {0, 0};  // S MMAs per query tile, over all pieces
        bool ok = true;
        for (int i = 0; ok; ++i) {
          if (!(ok = mbar_wait(&piece_full[i % kRing], (i / kRing) & 1, ctl))) break;
          const int n[2] = {pieces[i % kRing].n[0], pieces[i % kRing].n[1]};
          mbar_arrive(&piece_empty[i % kRing]);
          const int npos = positions<kTwin>(n[0], n[1]);
          if (npos < 0) break;
          if (npos == 0) continue;
          if (!(ok = mbar_wait(q_full, segs & 1, ctl))) break;
          ++segs;
          tc_fence_after();
          if constexpr (kTwin) {
            // the slots take turns: P V of a position follows its S by two
            for (int j = 0; j < npos + 2; ++j) {
              const int jg = base + j, s = jg % S, sp = (jg - 2 + S) % S, t = j & 1;
              if (j >= 2) {
                if (!(ok = mbar_wait(&v_full[sp], ((jg - 2) / S) & 1, ctl))) break;
                const int count = t == 0 ? issued[0] : issued[1];
                if (!(ok = mbar_wait(&p_full[t], (count - 1) & 1, ctl))) break;
                tc_fence_after();
                mma_ts_k128_step8(tmem + L::kColO0 + D * t, tmem + L::kColS0 + 128 * t,
                                  sdesc_sw128(sbase + L::kV + sp * L::kTile, 16384, 1024), idO,
                                  j >= 4 ? 1u : 0u);
                if (j >= npos) mma_commit(&o_full[t]);  // the slot's last P V
                mma_commit(&v_empty[sp]);
              }
              if (j < npos) {
                if (!(ok = mbar_wait(&k_full[s], (jg / S) & 1, ctl))) break;
                tc_fence_after();
                mma_ss_kmajor<D>(tmem + L::kColS0 + 128 * t,
                                 sdesc_sw128(sbase + L::kQ, 16384, 1024),
                                 sdesc_sw128(sbase + L::kK + s * L::kTile, 16384, 1024), idS, 0u);
                mma_commit(&s_full[t]);
                mma_commit(&k_empty[s]);
                issued[0] += 1 - t;
                issued[1] += t;
              }
            }
          } else {
            for (int j = 0; ok && j <= npos; ++j) {
              const int jg = base + j, s = jg % S, sp = (jg + S - 1) % S;
              if (j < npos && !(ok = mbar_wait(&k_full[s], (jg / S) & 1, ctl))) break;
              if (j >= 1 && !(ok = mbar_wait(&v_full[sp], ((jg - 1) / S) & 1, ctl))) break;
              tc_fence_after();
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                if (j >= 1 && j - 1 < n[t]) {
                  if (!(ok = mbar_wait(&p_full[t], (issued[t] - 1) & 1, ctl))) break;
                  tc_fence_after();
                  mma_ts_k128_step8(tmem + L::kColO0 + D * t, tmem + L::kColS0 + 128 * t,
                                    sdesc_sw128(sbase + L::kV + sp * L::kTile, 16384, 1024), idO,
                                    j > 1 ? 1u : 0u);
                  if (j == n[t]) mma_commit(&o_full[t]);  // the tile's last P V
                }
                if (j < n[t]) {  // S_t overwrites P_t: after the tile's own P V
                  mma_ss_kmajor<D>(tmem + L::kColS0 + 128 * t,
                                   sdesc_sw128(sbase + L::kQ + t * L::kTile, 16384, 1024),
                                   sdesc_sw128(sbase + L::kK + s * L::kTile, 16384, 1024), idS, 0u);
                  mma_commit(&s_full[t]);
                  ++issued[t];
                }
              }
              if (!ok) break;
              if (j < npos) mma_commit(&k_empty[s]);
              if (j >= 1) mma_commit(&v_empty[sp]);
            }
          }
          base += npos;
        }
        // every MMA issued by this thread has finished before tensor memory is released
        mma_commit(mma_done);
        drain_wait(mma_done, 0, ctl);
      }
    }
  } else {
    // ================= softmax warpgroups: one per query tile, one thread per row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int t = (warp - 4) >> 2;
    const uint32_t quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lanes = (quad * 32u) << 16;
    const uint32_t tS = tmem + lanes + L::kColS0 + 128 * t;
    const uint32_t tO = tmem + lanes + L::kColO0 + D * t;
    const uint32_t q_tile = sbase + L::kQ + t * L::kTile;
    const float c2 = a.scale_log2;
    int base = 0, segs = 0;  // positions and pieces with keys before this one
    int seen = 0, outs = 0;  // S tiles and results of this tile slot before this piece
    int twins = 0;           // twin pieces before this one
    bool ok = true;
    if (few_rows)
      rows16::work<D, kAllKeys>(a, l, part, rowbuf, shares[kLists == 2 ? warp - 4 : 0],
                                smem_u32(sm) + (warp - 4) * (rows16::PagedLayout<D>::kStages *
                                                             rows16::PagedLayout<D>::kStage),
                                nullptr, lane);
    for (int i = 0; !few_rows; ++i) {
      if (!(ok = mbar_wait_warp(&piece_full[i % kRing], (i / kRing) & 1, ctl))) break;
      const PieceInfo& piece = pieces[i % kRing];  // held until the piece is done
      const int n_mine = piece.n[t];
      if (n_mine < 0) break;
      const int npos = positions<kTwin>(piece.n[0], piece.n[1]);
      const int rows = piece.rows, r0 = piece.row0 + (kTwin ? 0 : 128 * t);  // r0: the tile's first row
      if (npos > 0) {
        // ---- the tile's queries: lanes 0-15 and 16-31 (d = 128) gather one row each time
        if (n_mine > 0 && !(kTwin && t == 1)) {
          constexpr int GR = D / 8, RI = 32 / GR;  // granules of a row, rows per step
          const int g = lane % GR;
          // lane i works out row i's place; two rounds of loads that are in flight together
          const int tok = (r0 + row) / a.G;
          const int place = r0 + row < rows ? (piece.start + tok) * a.H + piece.hk * a.G +
                                                  (r0 + row - tok * a.G)
                                            : -1;
#pragma unroll 1
          for (int k0 = 0; k0 < 32; k0 += 16) {
            uint4 v[16 / RI];
#pragma unroll
            for (int k = 0; k < 16 / RI; ++k) {
              const int at = __shfl_sync(~0u, place, k0 + k * RI + lane / GR);
              v[k] = make_uint4(0u, 0u, 0u, 0u);
              if (at >= 0)
                v[k] = *reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(at) * D + g * 8);
            }
#pragma unroll
            for (int k = 0; k < 16 / RI; ++k)
              st_shared_v4(q_tile + (g / 8) * 16384 +
                               sw128_offset(quad * 32 + k0 + k * RI + lane / GR, g % 8),
                           v[k].x, v[k].y, v[k].z, v[k].w);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();  // this warp's reads of the last piece's O precede its next MMAs
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        // no warp arrives for a later piece before every warp has for this one
        if (!(ok = mbar_wait_warp(q_full, segs & 1, ctl))) break;
        ++segs;
      }
      // keys below lim are visible to this row, and below lim_min to every row of the tile
      const int len = piece.len, ta = piece.ta;
      const int lim = l.causal && r0 + row < rows ? min(len, piece.shift + (r0 + row) / a.G + 1) : len;
      const int lim_min = M == kTreeKeys ? piece.shift
                                         : (l.causal ? min(len, piece.shift + r0 / a.G + 1) : len);
      // position whose last page ends inside it: that page's rows past the end are cleared
      const int tail = len & ((1 << a.page_shift) - 1), j_tail = tail != 0 ? len / KT - ta : -1;
      float m_run = -INFINITY, l_run = 0.f;
      for (int i_mine = 0; i_mine < n_mine; ++i_mine) {
        const int j = kTwin ? 2 * i_mine + t : i_mine, jg = base + j;
        if (!(ok = mbar_wait_warp(&s_full[t], (seen + i_mine) & 1, ctl))) break;
        tc_fence_after();
        uint32_t s[128];
        tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
        tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
        tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&s[64]));
        tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&s[96]));
        tmem_wait_ld();
        reg_fence(s);
        const int k0 = (ta + j) * KT;
        // hidden keys get a score of -inf in place, so that what follows is the same code for
        // every tile: it has to stay in the instruction cache next to the MMA issuer's loop
        if (k0 + KT > lim_min) {
          if constexpr (M == kTreeKeys) {
            const int tok = r0 + row < rows ? (r0 + row) / a.G : 0;
            const uint32_t* bits = a.tree + static_cast<int64_t>(piece.start + tok) * a.tree_words;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int left = len - k0 - 32 * x;  // keys of these 32 that there are
              uint32_t see = tree_window(bits, a.tree_words, k0 + 32 * x - lim_min);
              if (left < 32) see &= (1u << max(left, 0)) - 1u;
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!((see >> c) & 1u)) s[32 * x + c] = 0xff800000u;
            }
          } else {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (k0 + c >= lim) s[c] = 0xff800000u;
          }
        }
        float mxv[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
          mxv[0] = max3(mxv[0], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
          mxv[1] = max3(mxv[1], __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
          mxv[2] = max3(mxv[2], __uint_as_float(s[c + 4]), __uint_as_float(s[c + 5]));
          mxv[3] = max3(mxv[3], __uint_as_float(s[c + 6]), __uint_as_float(s[c + 7]));
        }
        const float mx = fmaxf(fmaxf(mxv[0], mxv[1]), fmaxf(mxv[2], mxv[3]));
        const float m_tile = mx * c2;
        float alpha = 1.f;
        bool rescale = false;
        // (whenever it grows, by however little: the row's largest weight is then exactly 1, and its
        // rounding to bf16 none; with 2^8 of slack O was off by up to twice as much at large logits, and the
        // trees above took 162.6 us)
        if (m_tile > m_run) {
          rescale = true;
          alpha = ex2(m_run - m_tile);  // 0 at the row's first visible key
          l_run *= alpha;
          m_run = m_tile;
        }
        const float2 cc = make_float2(c2, c2);
        const float neg = m_run == -INFINITY ? 0.f : -m_run;  // no visible key yet: all weights 0
        const float2 nm = make_float2(neg, neg);
        float2 sumv[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // weights in two halves of 64 keys, each stored over S as soon as it is packed (32 fewer
        // registers alive than with all of P).  c2 > 0, so -inf stays -inf and weighs 0.
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t p[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int k = 64 * hf + 2 * c;
            const float2 x = fma2(
                make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), cc, nm);
            const float x0 = ex2(x.x), x1 = ex2(x.y);
            p[c] = pack_bf16(x0, x1);
            sumv[c & 1] = add2(sumv[c & 1], make_float2(x0, x1));
          }
          tmem_st32(tS + 32 * hf, p);
        }
        l_run += (sumv[0].x + sumv[1].x) + (sumv[0].y + sumv[1].y);
        if (i_mine > 0 && __any_sync(0xffffffffu, rescale)) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
            tmem_wait_ld();
            reg_fence(o);
            const float2 aa = make_float2(alpha, alpha);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 v = mul2(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])),
                                    aa);
              o[i] = __float_as_uint(v.x);
              o[i + 1] = __float_as_uint(v.y);
            }
            tmem_st32(tO + 32 * c, o);
          }
        }
        // V rows of the last page past the end: cleared before this tile's P V may read them
        // (both warpgroups do, each before its own; zeros over zeros are harmless)
        if (j == j_tail) {
          if (!(ok = mbar_wait_warp(&v_full[jg % S], (jg / S) & 1, ctl))) break;
          const int past = len - k0, clear = ((1 << a.page_shift) - tail) * (D / 8);
          const uint32_t vt = sbase + L::kV + (jg % S) * L::kTile;
          for (int i = row; i < clear; i += 128) {
            const int rr = past + i / (D / 8), g = i % (D / 8);
            st_shared_v4(vt + (g / 8) * 16384 + rr * 128 + (g % 8) * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      seen += n_mine;
      base += npos;
      if (ok && n_mine > 0) ok = mbar_wait_warp(&o_full[t], outs++ & 1, ctl);
      if (!ok) break;
      tc_fence_after();
      // kTwin: slot 1 hands its statistics to slot 0, which joins the two results.  O of slot 1 and
      // the statistics stay until slot 0 has read them: the next piece's first MMA waits for all
      // warps on q_full
      float w0 = 1.f, w1 = 0.f;
      const bool both = kTwin && npos >= 2;  // slot 1 has had positions
      if (both) {
        if (t == 1) {
          twin_m[row] = m_run;
          twin_l[row] = l_run;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(twin_full);
        } else {
          if (!(ok = mbar_wait_warp(twin_full, twins++ & 1, ctl))) break;
          tc_fence_after();
          const float m1 = twin_m[row], l1 = twin_l[row], m = fmaxf(m_run, m1);
          // without a visible key a slot weighs nothing (NaN stays)
          w0 = m_run == -INFINITY ? (l_run == 0.f ? 0.f : l_run) : ex2(m_run - m);
          w1 = m1 == -INFINITY ? (l1 == 0.f ? 0.f : l1) : ex2(m1 - m);
          m_run = m;
          l_run = w0 * l_run + w1 * l1;
        }
      }

      // ---- this row's result, or its part of it
      const int gr = r0 + row;
      if (r0 < rows && !(kTwin && t == 1)) {  // uniform over the warpgroup
        const bool live = gr < rows;
        const int tok = gr / a.G, head = piece.hk * a.G + (gr - tok * a.G);
        const int64_t at = static_cast<int64_t>(piece.start + tok) * a.H + head;
        const bool final_out = piece.whole && rowbuf == nullptr;
        const float inv = l_run > 0.f ? 1.f / l_run : (l_run == 0.f ? 0.f : l_run);
        float* slot = part.slots + (static_cast<int64_t>(sh.worker) * 2 + (ta == 0 ? 1 : 0)) *
                                         (static_cast<int64_t>(R) * (D + 2));
        float* dst = piece.whole ? rowbuf + at * D : slot + (128 * t + row) * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (n_mine > 0) {
            tmem_ld32(tO + 32 * c, o);
            tmem_wait_ld();
            reg_fence(o);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
          if (both) {
            uint32_t o1[32];
            tmem_ld32(tO + D + 32 * c, o1);
            tmem_wait_ld();
            reg_fence(o1);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(fmaf(w1, __uint_as_float(o1[i]), w0 * __uint_as_float(o[i])));
          }
          if (!live) continue;
          if (final_out) {
            uint4* out = reinterpret_cast<uint4*>(a.o + at * D + 32 * c);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t pk[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                pk[i] = pack_bf16(__uint_as_float(o[8 * g + 2 * i]) * inv,
                                  __uint_as_float(o[8 * g + 2 * i + 1]) * inv);
              out[g] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
          } else {
#pragma unroll
            for (int g = 0; g < 4; ++g) st_v8(dst + 32 * c + 8 * g, &o[8 * g]);
          }
        }
        if (live) {
          if (final_out) {
            a.lse[static_cast<int64_t>(head) * a.total + piece.start + tok] =
                l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * kLn2;
          } else if (piece.whole) {
            float* st = rowbuf + static_cast<int64_t>(a.total) * a.H * D;
            st[at] = m_run;
            st[static_cast<int64_t>(a.total) * a.H + at] = l_run;
          } else {
            slot[R * D + 128 * t + row] = m_run;
            slot[R * D + R + 128 * t + row] = l_run;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&piece_empty[i % kRing]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

template <int D, int kLists, bool kTwin, KeyMode M>
cudaError_t launch_d(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a,
                     int64_t max_units, uint64_t timeout_ns, cudaStream_t s) {
  const uint32_t smem = smem_of<D, kLists>();  // the kernel's array is aligned as declared
  cudaError_t e = ensure_smem_limit<paged_mma_kernel<D, kLists, kTwin, M>>(smem);
  if (e != cudaSuccess) return e;
  const int64_t ctas = max_units < kPagedCtas ? max_units : kPagedCtas;
  return launch_chained(paged_mma_kernel<D, kLists, kTwin, M>, static_cast<unsigned>(ctas), kThreads,
                        smem, s, tk, tv, a, timeout_ns, smem);
}
template <int D>
cudaError_t launch_kind(KeyMode mode, const CUtensorMap& tk, const CUtensorMap& tv,
                        const PagedArgs& a, int lists, bool twin, int64_t max_units,
                        uint64_t timeout_ns, cudaStream_t s) {
  if (mode == kTreeKeys)
    return twin ? launch_d<D, 1, true, kTreeKeys>(tk, tv, a, max_units, timeout_ns, s)
                : launch_d<D, 1, false, kTreeKeys>(tk, tv, a, max_units, timeout_ns, s);
  if (lists == 2) return launch_d<D, 2, false, kAllKeys>(tk, tv, a, max_units, timeout_ns, s);
  return twin ? launch_d<D, 1, true, kAllKeys>(tk, tv, a, max_units, timeout_ns, s)
              : launch_d<D, 1, false, kAllKeys>(tk, tv, a, max_units, timeout_ns, s);
}

}  // namespace

cudaError_t launch_paged_mma(int d, KeyMode mode, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedArgs& a, int lists, bool twin, int64_t max_units,
                             uint64_t timeout_ns, cudaStream_t s) {
  return d == 64 ? launch_kind<64>(mode, tk, tv, a, lists, twin, max_units, timeout_ns, s)
                 : launch_kind<128>(mode, tk, tv, a, lists, twin, max_units, timeout_ns, s);
}

}  // namespace fa
