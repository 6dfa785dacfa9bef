// Launches of the attention of a few query rows (paged_rows.cuh), and the join of partial results.
#include "fa_internal.h"
#include "fa_paged.h"
#include "paged_plan.cuh"
#include "paged_rows.cuh"
#include "sm103.cuh"

namespace fa {

namespace {

constexpr int kWarps = kPagedWarps, kThreads = 32 * kWarps;
constexpr float kLn2 = 0.693147180559945309f;

// With two lists the CTAs are divided between them.
template <int D, int kLists>
__global__ void __launch_bounds__(kThreads, 1) paged_kernel(const __grid_constant__ PagedArgs a) {
  using rows16::KT;
  using rows16::R;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Share shares[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  touch(a);
  begin_launch();
  int li = 0;
  if constexpr (kLists == 1) {
    make_shares<R, KT, kThreads, kWarps>(a, shares);
  } else {
    __shared__ int red[2][3][kWarps], scan[kWarps];
    Entry mine[2];
    sum_entries<R, KT, kThreads>(a, a.list[0], mine[0], red[0]);
    sum_entries<R, KT, kThreads>(a, a.list[1], mine[1], red[1]);
    __syncthreads();
    const Totals t[2] = {totals_of(red[0]), totals_of(red[1])};
    const int n1 = ctas_of_second(a, gridDim.x, t), cta = blockIdx.x;
    li = cta < n1 ? 1 : 0;
    share_list<R, KT, kThreads, kWarps>(
        a, a.list[li], li ? t[1] : t[0], li ? mine[1] : mine[0], li ? cta : cta - n1,
        li ? n1 : static_cast<int>(gridDim.x) - n1, scan, shares);
  }
  rows16::work<D>(a, a.list[li], a.part[li], a.rowbuf[li], shares[warp],
                  smem_u32(smem) + warp * (rows16::PagedLayout<D>::kStages *
                                           rows16::PagedLayout<D>::kStage),
                  lane);
}

// Few segments, a CTA as the worker.  kPrefix: whole segments only, list 1 holds the prefixes.
template <int D, bool kPrefix>
__global__ void __launch_bounds__(kThreads, 1) paged_cta_kernel(const __grid_constant__ PagedArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Share shares[1];
  touch(a);
  begin_launch();
  make_shares<rows16::R, rows16::KT, kThreads, 1>(a, shares);
  if (kPrefix && blockIdx.x == 0)  // what is out of range in the groups is reported here
    for (int g = threadIdx.x; g < a.list[1].count; g += kThreads)
      entry_of<rows16::R, rows16::KT>(a.list[1], a, g, true);
  rows16::work_together<D, kPrefix>(a, a.list[0], a.part[0], shares[0], smem, threadIdx.x >> 5, threadIdx.x & 31);
}

// ---- join of the parts
constexpr int kJoinThreads = 128;
constexpr int kLanes = 8;                          // lanes of a group
constexpr int kGroups = kJoinThreads / kLanes;     // groups of a CTA

// O = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i over a row's parts, in the order of the keys.
// Bound by latency: spans, then m and l with the first parts of O, then the other parts.  kSplit
// groups of 8 lanes take every kSplit-th part of a row and meet in shared memory (the host chooses
// 1, 4 or 16 by the number of rows).
template <int D, int kSplit>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const JoinArgs a) {
  constexpr int E = D / kLanes / 4;  // float4s of a lane
  let_next_launch();
  constexpr int kRowsPerCta = kGroups / kSplit;
  constexpr int kDeep = kSplit == 1 ? 2 : 4;
  const int sub = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int crow = group / kSplit, pick = group % kSplit;  // row of the CTA, first part
  const unsigned mask = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
  const int rows = a.total * a.H;
  const int64_t id64 = static_cast<int64_t>(blockIdx.x) * kRowsPerCta + crow;
  const bool inside = id64 < rows;
  const int id = inside ? static_cast<int>(id64) : 0;
  const int t = id / a.H, head = id - t * a.H, hk = head / a.G;
  const int seq = token_sequence_group<kLanes>(a.cu, a.B, t, sub, mask);
  // where the row's parts are: its span and row tile in each list (these inputs are the call's)
  int where[2] = {-1, -1}, rr[2] = {0, 0};
  bool skip = !inside || seq < 0;
  for (int li = 0; li < a.lists && !skip; ++li) {
    const KeyList& l = a.list[li];
    int b = seq, start, n;
    if (l.group_cu != nullptr) {
      b = token_sequence_group<kLanes>(l.group_cu, l.count, seq, sub, mask);
      if (b < 0) continue;  // a sequence of no group has no prefix
      const int s0 = min(max(__ldg(l.group_cu + b), 0), a.B);
      start = a.cu != nullptr ? min(max(__ldg(a.cu + s0), 0), a.total) : s0;
      n = 0x7fffffff;
    } else {
      token_bounds(a.cu, b, a.total, start, n);
      n = min(n, l.max_q);
    }
    skip = t < start || t - start >= n;  // beyond max_q: not computed
    const int row = (t - start) * a.G + (head - hk * a.G);
    const int tile = row_tile0(start, a.G, a.part[li].R, b) + row / a.part[li].R;
    rr[li] = row % a.part[li].R;
    if (tile >= 0 && tile < a.part[li].span_tiles) where[li] = hk * a.part[li].span_tiles + tile;
  }
  wait_for_last_launch();
  float m = -INFINITY, lsum = 0.f;
  float4 o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  bool done = false;  // already final
  for (int li = 0; li < a.lists && !skip; ++li) {
    if (where[li] < 0) continue;
    const PartialLayout& p = a.part[li];
    const int2 span = p.spans[where[li]];
    if (!span_ok(span.x, span.y, p.workers)) continue;  // a launch that gave up left none
    const bool one = span.y == 1;
    if (one && a.rowbuf[li] == nullptr) {
      done = true;
      break;
    }
    const int64_t size = static_cast<int64_t>(p.R) * (D + 2);
    auto slot = [&](int i) { return p.slots + ((span.x + i) * 2 + (i == 0)) * size; };
    // this group's parts: i0, i0 + kSplit, ...; eight at a time, one lane each for m and l
    for (int i0 = pick; i0 < span.y; i0 += kLanes * kSplit) {
      const int mine = i0 + sub * kSplit, count = min(kLanes, (span.y - i0 + kSplit - 1) / kSplit);
      float pm = -INFINITY, pl = 0.f;
      if (mine < span.y) {
        const float* st = one ? a.rowbuf[li] + static_cast<int64_t>(rows) * D + id
                              : slot(mine) + p.R * D + rr[li];
        pm = st[0];
        pl = st[one ? rows : p.R];
      }
      // kDeep parts' O at a time, the first ones on the way together with m and l
      float4 v[kDeep][E];
      auto fetch = [&](int i, float4 (&to)[E]) {
        const float4* po = reinterpret_cast<const float4*>(
            one ? a.rowbuf[li] + static_cast<int64_t>(id) * D : slot(i0 + i * kSplit) + rr[li] * D);
#pragma unroll
        for (int e = 0; e < E; ++e)
          to[e] = i < count ? po[e * kLanes + sub] : make_float4(0.f, 0.f, 0.f, 0.f);
      };
#pragma unroll
      for (int k = 0; k < kDeep; ++k) fetch(k, v[k]);
      float top = pm;
#pragma unroll
      for (int x = kLanes / 2; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, x));
      top = fmaxf(top, m);
      const float keep = m == -INFINITY ? 0.f : ex2(m - top);
      // a part without a visible key has m = -inf and weighs nothing
      const float w = pm == -INFINITY ? (pl == 0.f ? 0.f : pl) : ex2(pm - top);
      float s = w * pl;
#pragma unroll
      for (int x = kLanes / 2; x > 0; x >>= 1) s += __shfl_xor_sync(mask, s, x);
      lsum = lsum * keep + s;
      m = top;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        o[e].x *= keep; o[e].y *= keep; o[e].z *= keep; o[e].w *= keep;
      }
      for (int i = 0; i < count; i += kDeep) {
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
          const float wi = __shfl_sync(mask, w, i + k, kLanes);  // 0 past the last part
          if (i + k >= count) break;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            o[e].x = fmaf(wi, v[k][e].x, o[e].x);
            o[e].y = fmaf(wi, v[k][e].y, o[e].y);
            o[e].z = fmaf(wi, v[k][e].z, o[e].z);
            o[e].w = fmaf(wi, v[k][e].w, o[e].w);
          }
          if (i + k + kDeep < count) fetch(i + k + kDeep, v[k]);
        }
      }
    }
  }
  if constexpr (kSplit > 1) {
    __shared__ float4 so[kGroups][D / 4];
    __shared__ float sm[kGroups], sl[kGroups];
#pragma unroll
    for (int e = 0; e < E; ++e) so[group][e * kLanes + sub] = o[e];
    if (sub == 0) {
      sm[group] = m;
      sl[group] = lsum;
    }
    __syncthreads();
    if (pick != 0) return;
    m = -INFINITY;
    lsum = 0.f;
#pragma unroll
    for (int g = 0; g < kSplit; ++g) m = fmaxf(m, sm[group + g]);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g = 0; g < kSplit; ++g) {
      const float gm = sm[group + g], gl = sl[group + g];
      const float w = gm == -INFINITY ? (gl == 0.f ? 0.f : gl) : ex2(gm - m);
      lsum = fmaf(w, gl, lsum);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float4 v = so[group + g][e * kLanes + sub];
        o[e].x = fmaf(w, v.x, o[e].x);
        o[e].y = fmaf(w, v.y, o[e].y);
        o[e].z = fmaf(w, v.z, o[e].z);
        o[e].w = fmaf(w, v.w, o[e].w);
      }
    }
  }
  if (skip || done) return;
  const float inv = lsum > 0.f ? 1.f / lsum : (lsum == 0.f ? 0.f : lsum);
  uint2* dst = reinterpret_cast<uint2*>(a.o + static_cast<int64_t>(id) * D);
#pragma unroll
  for (int e = 0; e < E; ++e)
    dst[e * kLanes + sub] = make_uint2(pack_bf16(o[e].x * inv, o[e].y * inv),
                                       pack_bf16(o[e].z * inv, o[e].w * inv));
  if (sub == 0)
    a.lse[static_cast<int64_t>(head) * a.total + t] =
        lsum == 0.f ? -INFINITY : (m + log2f(lsum)) * kLn2;
}

template <int D, int kLists>
cudaError_t launch_paged_d(const PagedArgs& a, int64_t max_units, cudaStream_t s) {
  constexpr uint32_t bytes = rows16::PagedLayout<D>::kBytes;
  cudaError_t e = ensure_smem_limit<paged_kernel<D, kLists>>(bytes);
  if (e != cudaSuccess) return e;
  const int64_t ctas = max_units < kPagedCtas ? max_units : kPagedCtas;
  return launch_chained(paged_kernel<D, kLists>, static_cast<unsigned>(ctas), kThreads, bytes, s, a);
}

template <int D, bool kPrefix>
cudaError_t launch_cta_d(const PagedArgs& a, int64_t max_units, cudaStream_t s) {
  constexpr uint32_t bytes = rows16::PagedLayout<D>::kBytes;
  cudaError_t e = ensure_smem_limit<paged_cta_kernel<D, kPrefix>>(bytes);
  if (e != cudaSuccess) return e;
  const int64_t ctas = max_units < kPagedCtas ? max_units : kPagedCtas;
  return launch_chained(paged_cta_kernel<D, kPrefix>, static_cast<unsigned>(ctas), kThreads, bytes,
                        s, a);
}

template <int D>
cudaError_t launch_join_d(const JoinArgs& a, int split, cudaStream_t s) {
  const unsigned rows = static_cast<unsigned>(a.total) * static_cast<unsigned>(a.H);
  const unsigned per = kGroups / split, grid = (rows + per - 1) / per;
  if (split == 16) return launch_chained(paged_join_kernel<D, 16>, grid, kJoinThreads, 0, s, a);
  if (split == 4) return launch_chained(paged_join_kernel<D, 4>, grid, kJoinThreads, 0, s, a);
  return launch_chained(paged_join_kernel<D, 1>, grid, kJoinThreads, 0, s, a);
}

}  // namespace

cudaError_t launch_paged(int d, const PagedArgs& a, int lists, int64_t max_units, cudaStream_t s) {
  if (lists == 2)
    return d == 64 ? launch_paged_d<64, 2>(a, max_units, s)
                   : launch_paged_d<128, 2>(a, max_units, s);
  return d == 64 ? launch_paged_d<64, 1>(a, max_units, s) : launch_paged_d<128, 1>(a, max_units, s);
}

cudaError_t launch_paged_cta(int d, const PagedArgs& a, int lists, int64_t max_units,
                             cudaStream_t s) {
  if (lists == 2)
    return d == 64 ? launch_cta_d<64, true>(a, max_units, s)
                   : launch_cta_d<128, true>(a, max_units, s);
  return d == 64 ? launch_cta_d<64, false>(a, max_units, s)
                 : launch_cta_d<128, false>(a, max_units, s);
}

cudaError_t launch_paged_join(int d, const JoinArgs& a, int split, cudaStream_t s) {
  return d == 64 ? launch_join_d<64>(a, split, s) : launch_join_d<128>(a, split, s);
}

}  // namespace fa
