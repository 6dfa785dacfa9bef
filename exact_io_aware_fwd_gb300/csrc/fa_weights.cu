// Attention weights of the keys of a paged cache, summed over queries, on the tcgen05 tensor cores.
//
//   out_j = in_j + sum over a key/value head's queries of exp(scale q.k_j - LSE)
//
// the probabilities that attention used, from the LSE it left: one product instead of two, and no
// maximum to keep.  Keys are the rows of the product and queries its columns, S^T = K Q^T, so that a
// thread owns a key: it adds up its row of tensor memory, and nothing is exchanged or joined.  Bound
// by reading the keys once (256 flops a 2-byte element at 128 queries, half of what the tensor core
// has per byte), so one kernel serves single tokens and windows of them: one token of 64 sequences of 512
// to 4096 keys, 8 heads, d = 128, 56.5 us (5.4 TB/s), 32 tokens of 8 sequences of 16384 keys 40.7 us (5.3
// TB/s, the tensor core 30% busy); 131072 keys run at the rate of a copy.  What is missing is the start
// (1.8 us until a CTA knows its share, 1.9 until its first copy, 1.5 until that is there) and CTAs that
// end up to 5 us apart.
//
// CTAs are persistent and take equal shares of all key tiles (paged_plan.cuh).  Warp 2 works out a
// CTA's pieces and hands them to the others through a ring; a piece is worked on once for every 128
// queries (a job), the sums of the later ones on top of the earlier ones' (in global memory, by the
// same threads).  The warpgroups of a CTA take key tiles in turn, each with a buffer of tensor memory,
// and write the next job's queries into shared memory before they turn to this one's tiles.  Warp 3
// copies what no query sees.
#include "fa_cache.h"
#include "fa_internal.h"
#include "paged_plan.cuh"
#include "sm103.cuh"

namespace fa {

namespace {

constexpr int kGroups = 2;  // warpgroups of weights (four: 43.0 us for 8 x 32 tokens over 16384 keys, two: 41.4)
constexpr int kWarps = 4 * kGroups;
constexpr int kThreads = 128 + 32 * kWarps;  // warp 0: TMA, 1: MMA, 2: pieces, 3: columns past the keys
constexpr int KT = 128;        // keys of a tile
constexpr int kAllRows = 1 << 30;  // the plan knows one row tile: a piece has all of its queries
constexpr int NQ = 128;        // queries of a job
constexpr int kRing = 4;
constexpr int kStats = 4;  // jobs whose queries' statistics are kept: a warp may be three ahead of another
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void prefetch_l1(const void* p) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(p) : "memory");
}

struct PieceInfo {
  int n;            // key tiles; -1: no more pieces
  int ta;           // first key tile
  int bh, hk;       // row of `out`, key/value head
  int start, rows;  // the sequence's first token and its queries (computed tokens x group)
  int len, shift;   // keys, and keys minus tokens
  const int32_t* table;
};

template <int D>
struct Layout {
  static constexpr uint32_t kTile = 128u * D * 2u;
  static constexpr int kStages = D == 128 ? 4 : 8;  // 128 KB on the way
  static constexpr uint32_t kK = 0, kQ = kStages * kTile, kBytes = kQ + 2 * kTile;
  static constexpr uint32_t kTmemCols = NQ * kGroups;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ PagedArgs a,
                   const __grid_constant__ WeightsOut w, const uint64_t timeout_ns) {
  using L = Layout<D>;
  constexpr int S = L::kStages, P = D / 64;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ uint64_t k_full[S], k_empty[S], q_full[2], q_empty[2], s_full[kGroups], s_empty[kGroups],
      mma_done[1];
  __shared__ uint64_t piece_full[kRing], piece_empty[kRing];
  __shared__ PieceInfo pieces[kRing];
  __shared__ alignas(16) float less[kStats][NQ];  // -LSE in log2 units of a job's queries
  __shared__ int sees[kStats][NQ];    // keys below it are visible
  __shared__ uint32_t tmem_slot[1];
  __shared__ volatile int abort_flag[1];
  __shared__ Share shares[1];
  const Ctl ctl{abort_flag, a.status, timeout_ns};
  const uint32_t warp = warp_id(), lane = lane_id();
  if ((smem_u32(sm) & 1023u) != 0) {  // cannot happen: the array is aligned; never proceed
    if (threadIdx.x == 0) atomicCAS(a.status, 0, kErrLayout);
    return;
  }
  if (warp == 0 && lane == 0) {
    *abort_flag = 0;
    for (int s = 0; s < S; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], kWarps);
      mbar_init(&q_empty[t], 1);
    }
    for (int t = 0; t < kGroups; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&s_empty[t], 4);
    }
    mbar_init(mma_done, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], 2 + kWarps);  // TMA warp, MMA thread, warps of weights
    }
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  touch(a);
  begin_launch();
  make_shares<kAllRows, KT, kThreads, 1>(a, shares);
  const KeyList& l = a.list[0];
  const uint32_t tmem = *tmem_slot, sbase = smem_u32(sm);
  if (warp == 2) {
    // ================= the CTA's pieces
    if (lane == 0) {
      Walk<kAllRows, KT> walk(a, l, shares[0]);
      const Entry& e = walk.e;
      Piece piece;
      int n = 0;  // key tiles; none of a sequence without keys, or behind the last key
      for (int i = 0;; ++i) {
        bool more;
        while ((more = walk.next(a, l, piece)) && (n = min(piece.te, (e.len + KT - 1) / KT) - piece.ta) <= 0) {
        }
        if (!mbar_wait(&piece_empty[i % kRing], ((i / kRing) & 1) ^ 1, ctl)) break;
        PieceInfo& p = pieces[i % kRing];
        if (more) {
          prefetch_l1(l.table + static_cast<int64_t>(walk.b) * l.max_pages + (piece.ta << 7 >> a.page_shift));
          p.n = n;
          p.ta = piece.ta;
          p.bh = walk.b * a.Hkv + piece.hk;
          p.hk = piece.hk;
          p.start = e.start;
          p.rows = e.nc * a.G;
          p.len = e.len;
          p.shift = e.len - e.n;
          p.table = l.table + static_cast<int64_t>(walk.b) * l.max_pages;
        } else {
          p.n = -1;
        }
        mbar_arrive(&piece_full[i % kRing]);
        if (!more) break;
      }
    }
  } else if (warp == 3) {
    // ================= columns that no query sees: what there was
    if (w.in != w.out) {
      for (int bh = blockIdx.x; bh < a.B * a.Hkv; bh += gridDim.x) {
        const Entry e = entry_of<kAllRows, KT>(l, a, bh / a.Hkv, false);
        const int64_t row = static_cast<int64_t>(bh) * w.cap;
        constexpr int kAhead = 16;
        for (int j0 = (e.nc > 0 ? e.len : 0) + lane; j0 < w.cap; j0 += 32 * kAhead) {
          float v[kAhead];
#pragma unroll
          for (int i = 0; i < kAhead; ++i)
            v[i] = w.in != nullptr && j0 + 32 * i < w.cap ? w.in[row + j0 + 32 * i] : 0.f;
#pragma unroll
          for (int i = 0; i < kAhead; ++i)
            if (j0 + 32 * i < w.cap) w.out[row + j0 + 32 * i] = v[i];
        }
      }
    }
  } else if (warp == 0) {
    // ================= TMA producer: one box (page x 64 columns) per lane
    const int page_size = 1 << a.page_shift, pages = KT >> a.page_shift;
    const int pg = lane & (pages - 1), panel = lane / pages;
    int jk = 0;  // tiles whose copies have been issued
    // page of this lane's box at key tile kt: the map's out-of-range coordinate, which reads as zeros,
    // past the end and (reported) for a page outside the pool
    auto find = [&](const PieceInfo& p, int kt) {
      const int key = kt * KT + pg * page_size;
      if (key >= p.len) return a.num_pages * a.Hkv;
      const int page = resolve_page(p.table, l.max_pages, a.num_pages, a.page_shift, key);
      if (page < 0) atomicCAS(a.status, 0, kErrIndex);
      return page < 0 ? a.num_pages * a.Hkv : page * a.Hkv + p.hk;
    };
    auto take = [&](int i, PieceInfo& p) {
      if (!mbar_wait_warp(&piece_full[i % kRing], (i / kRing) & 1, ctl)) return false;
      p = pieces[i % kRing];
      __syncwarp();
      if (lane == 0) mbar_arrive(&piece_empty[i % kRing]);  // all of it is in registers
      return true;
    };
    PieceInfo p;
    bool ok = take(0, p);
    int z_next = ok && p.n > 0 ? find(p, p.ta) : 0;
    for (int i = 1; ok && p.n > 0; ++i) {
      PieceInfo q;  // the piece behind this one
      const int jobs = (p.rows + NQ - 1) / NQ;
      for (int r = 0; ok && r < jobs; ++r) {
        for (int j = 0; j < p.n; ++j, ++jk) {
          const int s = jk % S, z = z_next;
          if (j + 1 < p.n) {
            z_next = find(p, p.ta + j + 1);
          } else if (r + 1 < jobs) {
            z_next = find(p, p.ta);
          } else {
            if (!(ok = take(i, q))) break;
            z_next = q.n > 0 ? find(q, q.ta) : 0;
          }
          if (!(ok = mbar_wait_warp(&k_empty[s], ((jk / S) & 1) ^ 1, ctl))) break;
          if (lane == 0) mbar_arrive_expect_tx(&k_full[s], L::kTile);
          __syncwarp();
          // the block table's next line, so that finding a page does not hold up the copies
          if (lane == 0) prefetch_l1(p.table + min(((p.ta + j + 1) << 7 >> a.page_shift) + 32, l.max_pages - 1));
          if (panel < P)
            tma_load_3d(sm + L::kK + s * L::kTile + panel * 16384 + pg * (page_size * 128), &tmK, &k_full[s],
                        panel * 64, 0, z);
        }
      }
      p = q;
    }
    // no copy into this CTA's shared memory may still be in flight when the CTA exits
    if (lane == 0)
      for (int j = max(0, jk - S); j < jk; ++j) drain_wait(&k_full[j % S], (j / S) & 1, ctl);
  } else if (warp == 1) {
    // ================= MMA issuer
    if (lane == 0) {
      int jk = 0, jobs = 0;
      uint32_t turns = 0;  // bit t: an odd number of products into buffer t
      bool ok = true;
      for (int i = 0; ok; ++i) {
        if (!(ok = mbar_wait(&piece_full[i % kRing], (i / kRing) & 1, ctl))) break;
        const int n = pieces[i % kRing].n, rows = pieces[i % kRing].rows;
        mbar_arrive(&piece_empty[i % kRing]);
        if (n < 0) break;
        for (int r = 0; ok && r * NQ < rows; ++r, ++jobs) {
          const int slot = jobs & 1;
          if (!(ok = mbar_wait(&q_full[slot], (jobs >> 1) & 1, ctl))) break;
          // columns in steps of 16, as the instruction takes them
          const uint32_t id = idesc_bf16(128, (min(NQ, rows - r * NQ) + 15) / 16 * 16, false, false);
          for (int j = 0; j < n; ++j, ++jk) {
            const int s = jk % S, t = j % kGroups;
            if (!(ok = mbar_wait(&k_full[s], (jk / S) & 1, ctl))) break;
            if (!(ok = mbar_wait(&s_empty[t], (turns >> t & 1) ^ 1, ctl))) break;
            tc_fence_after();
            mma_ss_kmajor<D>(tmem + NQ * t, sdesc_sw128(sbase + L::kK + s * L::kTile, 16384, 1024),
                             sdesc_sw128(sbase + L::kQ + slot * L::kTile, 16384, 1024), id, 0u);
            mma_commit(&s_full[t]);
            mma_commit(&k_empty[s]);
            turns ^= 1u << t;
          }
          if (ok) mma_commit(&q_empty[slot]);
        }
      }
      // every MMA issued by this thread has finished before tensor memory is released
      mma_commit(mma_done);
      drain_wait(mma_done, 0, ctl);
    }
  } else {
    // ================= weights: one thread per key of a tile
    const int t = (warp - 4) >> 2, quad = warp & 3;
    const uint32_t tS = tmem + ((quad * 32u) << 16) + NQ * t;
    const float2 c2 = make_float2(a.scale_log2, a.scale_log2);
    int jobs = 0, seen = 0;  // jobs before this one, tiles of this warpgroup's buffer
    struct Job {
      int i, r;  // piece, and which 128 of its queries
    };
    auto live = [&](const Job& j) { return pieces[j.i % kRing].n > 0; };
    auto next_job = [&](Job& j) {  // false: gave up
      if ((j.r + 1) * NQ < pieces[j.i % kRing].rows) {
        ++j.r;
        return true;
      }
      ++j.i;
      j.r = 0;
      return mbar_wait_warp(&piece_full[j.i % kRing], (j.i / kRing) & 1, ctl);
    };
    // Some of a job's queries and their statistics: loaded one job before they are written to the job's
    // slot, which is one job before it is their turn
    constexpr int GR = D / 8, RI = 32 / GR, QW = NQ / kWarps;  // granules of a row, rows per step and warp
    static_assert(QW >= RI && QW <= 32, "whole steps");
    const int q0 = (warp - 4) * QW;
    uint4 v[QW / RI];
    float stat = 0.f;
    int limit = 0;
    bool any = false;  // this warp has queries of the job
    auto fetch = [&](const Job& j) {
      const PieceInfo& p = pieces[j.i % kRing];
      const int rows = min(NQ, p.rows - j.r * NQ), mine = q0 + (lane & (QW - 1)), row = j.r * NQ + mine, tok = row / a.G;
      const int head = p.hk * a.G + (row - tok * a.G);
      const int place = mine < rows ? (p.start + tok) * a.H + head : -1;
      any = q0 < (rows + 15) / 16 * 16;  // what the product takes
      if (!any) return;
      stat = -INFINITY;  // the LSE of a row without keys, or of no row
      limit = 0;
      if (lane < QW && place >= 0) {
        stat = w.lse[static_cast<int64_t>(head) * a.total + p.start + tok];
        limit = w.causal ? min(p.len, p.shift + tok + 1) : p.len;
      }
#pragma unroll
      for (int k = 0; k < QW / RI; ++k) {
        const int from = __shfl_sync(~0u, place, k * RI + lane / GR);
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (from >= 0)
          v[k] = *reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(from) * D + (lane % GR) * 8);
      }
    };
    auto put = [&](int job) {  // false: gave up
      if (!mbar_wait_warp(&q_empty[job & 1], ((job >> 1) & 1) ^ 1, ctl)) return false;
      if (any) {
        const uint32_t q_tile = sbase + L::kQ + (job & 1) * L::kTile;
        if (lane < QW) {
          less[job % kStats][q0 + lane] = stat == -INFINITY ? -INFINITY : -stat * kLog2e;  // weighs nothing
          sees[job % kStats][q0 + lane] = limit;
        }
#pragma unroll
        for (int k = 0; k < QW / RI; ++k)
          st_shared_v4(q_tile + (lane % GR / 8) * 16384 + sw128_offset(q0 + k * RI + lane / GR, lane % 8), v[k].x,
                       v[k].y, v[k].z, v[k].w);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[job & 1]);
      return true;
    };
    // What this thread's key of the job's tile j had before; loaded a tile ahead.
    auto had = [&](const Job& job, int j) {
      const PieceInfo& p = pieces[job.i % kRing];
      const int key = (p.ta + j) * KT + quad * 32 + lane;
      const float* const from = job.r > 0 ? w.out : w.in;
      return j < p.n && key < p.len && from != nullptr ? from[static_cast<int64_t>(p.bh) * w.cap + key] : 0.f;
    };
    float ahead = 0.f;
    Job cur{0, 0}, behind{0, 0};
    bool ok = mbar_wait_warp(&piece_full[0], 0, ctl);
    if (ok && live(cur)) {
      fetch(cur);
      ahead = had(cur, t);
      ok = put(0) && next_job(behind);
      if (ok && live(behind)) fetch(behind);
    }
    while (ok && live(cur)) {
      const PieceInfo& p = pieces[cur.i % kRing];  // held until its last job is done
      const int r = cur.r;
      Job far = behind;
      if (live(behind)) {
        if (!(ok = put(jobs + 1) && next_job(far))) break;
        if (live(far)) fetch(far);
      }
      if (!(ok = mbar_wait_warp(&q_full[jobs & 1], (jobs >> 1) & 1, ctl))) break;  // and their statistics
      const int rows = min(NQ, p.rows - r * NQ), len = p.len;
      const float* const off = less[jobs % kStats];
      const int* const lim = sees[jobs % kStats];
      const int all = w.causal ? min(len, p.shift + r * NQ / a.G + 1) : len;  // keys that every query sees
      const int64_t line = static_cast<int64_t>(p.bh) * w.cap;
      bool left_out = false;  // a query with an LSE of -inf: its scores may be anything
#pragma unroll
      for (int c = 0; c < NQ; c += 32)
        if (c + static_cast<int>(lane) < rows) left_out |= off[c + lane] == -INFINITY;
      left_out = __any_sync(~0u, left_out);
      float next = r > 0 ? had(cur, t) : ahead;
      if (live(behind) && behind.r == 0) ahead = had(behind, t);
      for (int j = t; j < p.n; j += kGroups) {
        const int k0 = (p.ta + j) * KT, key = k0 + quad * 32 + lane;
        const float was = next;
        next = had(cur, j + kGroups);
        if (!(ok = mbar_wait_warp(&s_full[t], seen++ & 1, ctl))) break;
        tc_fence_after();
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const bool masked = w.causal && k0 + KT > all;
#pragma unroll 1
        for (int c = 0; c < rows; c += 32) {
          uint32_t s[32];
          tmem_ld32(tS + c, s);
          tmem_wait_ld();
          reg_fence(s);
          if (c + 32 >= rows) {  // all of it has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[t]);
          }
          if (left_out) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (off[c + k] == -INFINITY) s[k] = 0u;
          }
          if (!masked && c + 32 <= rows) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 o = *reinterpret_cast<const float4*>(off + c + k);
              const float2 x = fma2(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), c2,
                                    make_float2(o.x, o.y));
              const float2 y = fma2(make_float2(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])), c2,
                                    make_float2(o.z, o.w));
              sum[0] = add2(sum[0], make_float2(ex2(x.x), ex2(x.y)));
              sum[1] = add2(sum[1], make_float2(ex2(y.x), ex2(y.y)));
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const bool there = c + k < rows && key < lim[min(c + k, NQ - 1)];
              const float p1 = ex2(fmaf(__uint_as_float(s[k]), a.scale_log2, off[min(c + k, NQ - 1)]));
              if (there) sum[(k >> 1) & 1].x += p1;
            }
          }
        }
        if (key < len) w.out[line + key] = was + ((sum[0].x + sum[1].x) + (sum[0].y + sum[1].y));
      }
      if (!ok) break;
      ++jobs;
      if (behind.i != cur.i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&piece_empty[cur.i % kRing]);
      }
      cur = behind;
      behind = far;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

template <int D>
cudaError_t launch_d(const CUtensorMap& tk, const PagedArgs& a, const WeightsOut& w, uint64_t timeout_ns,
                     cudaStream_t s) {
  const cudaError_t e = ensure_smem_limit<weights_kernel<D>>(Layout<D>::kBytes);
  if (e != cudaSuccess) return e;
  return launch_chained(weights_kernel<D>, static_cast<unsigned>(kPagedCtas), kThreads, Layout<D>::kBytes, s, tk, a,
                        w, timeout_ns);
}

}  // namespace

cudaError_t launch_kv_weights(int d, const CUtensorMap& tk, const PagedArgs& a, const WeightsOut& w,
                              uint64_t timeout_ns, cudaStream_t s) {
  return d == 64 ? launch_d<64>(tk, a, w, timeout_ns, s) : launch_d<128>(tk, a, w, timeout_ns, s);
}

}  // namespace fa
