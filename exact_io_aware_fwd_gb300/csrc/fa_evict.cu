// Attention weights summed over queries, and the eviction of the keys that have gathered least.
#include "fa_cache.h"
#include "fa_internal.h"
#include "paged_rows.cuh"
#include "select_kth.cuh"
#include "sm103.cuh"

namespace fa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ---- weights
// out_j = in_j + sum over a key/value head's queries of exp(scale q.k_j - LSE): the probabilities
// that attention used, from the LSE it left, so one product instead of two and no maximum to keep.
// Keys do not depend on each other: a warp takes 32 of them as the columns of an m16n8k16 product
// and goes through the query rows 16 at a time; what a lane adds up stays its own until the end.
// Keys are loaded 16 bytes a lane straight into fragments (page_score_kernel's order of k).
constexpr int kWeightWarps = 4, kWeightKeys = 32;

template <int D>
__global__ void __launch_bounds__(32 * kWeightWarps) kv_weights_kernel(const WeightsArgs a, int chunks) {
  constexpr int J = D / 32, T = kWeightKeys / 8;
  begin_launch();
  const CacheSeqs& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = static_cast<int>(blockIdx.x) / chunks, chunk = static_cast<int>(blockIdx.x) % chunks;
  const int b = bh / c.Hkv, hk = bh - b * c.Hkv;
  const int k0 = (chunk * kWeightWarps + warp) * kWeightKeys;
  if (k0 >= a.cap) return;
  const int len = keys_of(c, b, threadIdx.x == 0 && chunk == 0 && hk == 0);
  const int64_t row = static_cast<int64_t>(bh) * a.cap;
  if (k0 >= len) {  // no keys: what there was
    const int key = k0 + lane;
    if (a.in != a.out && key < a.cap) a.out[row + key] = a.in != nullptr ? a.in[row + key] : 0.f;
    return;
  }
  int start, n;
  token_bounds(c.cu, b, c.total, start, n);
  const int nc = min(n, a.max_q);
  if (nc < n && threadIdx.x == 0 && chunk == 0 && hk == 0) atomicCAS(c.status, 0, kErrIndex);
  uint4 kf[T][J];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int key = k0 + 8 * t + (lane >> 2);
    const int phys = key < len ? page_of(c, b, key >> c.page_shift) : -1;
    const uint4* src = reinterpret_cast<const uint4*>(
                           a.k_cache + (((static_cast<int64_t>(max(phys, 0)) * c.Hkv + hk) << c.page_shift) +
                                        (key & ((1 << c.page_shift) - 1))) * D) + (lane & 3);
#pragma unroll
    for (int j = 0; j < J; ++j) kf[t][j] = phys >= 0 ? __ldg(src + 4 * j) : make_uint4(0u, 0u, 0u, 0u);
  }
  float sum[T][2] = {};
  const int rows = nc * a.G, shift = len - n;
  for (int r0 = 0; r0 < rows; r0 += 16) {
    const uint4* q[2];
    float off[2];  // LSE in log2 units
    int lim[2];    // keys below it are visible to the row
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rr = r0 + (lane >> 2) + 8 * i;
      const bool live = rr < rows;
      const int tok = live ? rr / a.G : 0, head = hk * a.G + (live ? rr - tok * a.G : 0);
      q[i] = reinterpret_cast<const uint4*>(a.q + (static_cast<int64_t>(start + tok) * a.H + head) * D) + (lane & 3);
      const float lse = __ldg(a.lse + static_cast<int64_t>(head) * c.total + start + tok);
      off[i] = lse == -INFINITY ? INFINITY : lse * kLog2e;  // a row without keys weighs nothing
      lim[i] = !live ? 0 : (a.causal ? min(len, shift + tok + 1) : len);
    }
    float s[T][4];
#pragma unroll
    for (int t = 0; t < T; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint4 v0 = __ldg(q[0] + 4 * j), v1 = __ldg(q[1] + 4 * j);
      const uint32_t f0[4] = {v0.x, v1.x, v0.y, v1.y}, f1[4] = {v0.z, v1.z, v0.w, v1.w};
#pragma unroll
      for (int t = 0; t < T; ++t) {
        rows16::mma16816(s[t], f0, kf[t][j].x, kf[t][j].y);
        rows16::mma16816(s[t], f1, kf[t][j].z, kf[t][j].w);
      }
    }
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = k0 + 8 * t + (lane & 3) * 2 + (k & 1);
        const float p = ex2(fmaf(s[t][k], a.scale_log2, -off[k >> 1]));
        if (key < lim[k >> 1]) sum[t][k & 1] += p;
      }
  }
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum[t][k] += __shfl_xor_sync(~0u, sum[t][k], o);
  // lane l writes key l: column l % 8 of tile l / 8 is with the lanes of (l % 8) / 2
  float mine = 0.f;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const float x = __shfl_sync(~0u, sum[t][0], (lane & 7) >> 1), y = __shfl_sync(~0u, sum[t][1], (lane & 7) >> 1);
    if (lane >> 3 == t) mine = lane & 1 ? y : x;
  }
  const int key = k0 + lane;
  if (key < a.cap) {
    const float was = a.in != nullptr ? a.in[row + key] : 0.f;
    a.out[row + key] = key < len ? was + mine : was;
  }
}

// ---- eviction: which keys stay
// The smallest weight that stays by counting (select_kth.cuh), then the keys in order.  A sequence
// and head is a CTA's, or, where a CTA's registers (kRounds weights a thread) do not hold its
// weights, a cluster's, each CTA with a stretch of them; only what does not fit eight CTAs is read
// again in every pass.
constexpr int kRounds = 16;
constexpr int evict_cluster(int max_len, int threads) {
  int c = 1;
  while (c < 8 && c * kRounds * threads < max_len) c *= 2;
  return c;
}

template <int kThreads, bool kCluster>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ KthShared<kThreads, uint32_t> sh;
  __shared__ OrderShared<kThreads, kRounds> order_sh;
  __shared__ alignas(8) unsigned totals[2];  // above the k-th, in its range
  begin_launch();
  const CacheSeqs& c = a.c;
  const int rank = kCluster ? cluster_rank() : 0, ctas = kCluster ? cluster_size() : 1;
  const int row = static_cast<int>(blockIdx.x) / ctas, tid = threadIdx.x, all = rank * kThreads + tid;
  const int b = row / c.Hkv, hk = row - b * c.Hkv;
  const int len = keys_of(c, b, all == 0 && hk == 0);
  const int count = min(len, a.budget);
  if (all == 0 && hk == 0) a.new_lens[b] = count;
  const float* w = a.weights + static_cast<int64_t>(row) * a.cap;
  int32_t* kept = a.kept + static_cast<int64_t>(row) * a.budget;
  float* left = a.new_weights + static_cast<int64_t>(row) * a.budget;
  const int old = len > a.budget ? len - a.recent : 0;  // keys that are chosen from
  const int k = count - (len - old);                    // and how many of them stay
  // this CTA's stretch, its first kRounds rounds in registers
  const int chunk = (old + ctas - 1) / ctas, c0 = min(old, rank * chunk), c1 = min(old, c0 + chunk);
  float x[kRounds];
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int at = c0 + i * kThreads + tid;
    x[i] = at < c1 ? w[at] : 0.f;
  }
  for (int i = count + all; i < a.budget; i += ctas * kThreads) {
    kept[i] = -1;
    left[i] = 0.f;
  }
  for (int i = old + all; i < len; i += ctas * kThreads) {
    kept[k + i - old] = i;
    left[k + i - old] = w[i];
  }
  if (k == 0) return;  // the whole cluster
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      if (c0 + i * kThreads + tid < c1) f(ordered(x[i]));
    for (int at = c0 + kRounds * kThreads + tid; at < c1; at += kThreads) f(ordered(w[at]));
  };
  const Kth<uint32_t> kth = kth_largest<kThreads, kCluster, uint32_t>(k, 32, each, sh);
  unsigned over0 = 0, tie0 = 0;  // in front of this CTA's stretch
  if constexpr (kCluster) {
    if (tid == 0) totals[0] = totals[1] = 0;
    __syncthreads();
    unsigned over = 0, tie = 0;
    each([&](uint32_t key) {
      over += kth.under(key);
      tie += kth.holds(key);
    });
    over = __reduce_add_sync(~0u, over);
    tie = __reduce_add_sync(~0u, tie);
    if ((tid & 31) == 0) {
      atomicAdd(&totals[0], over);
      atomicAdd(&totals[1], tie);
    }
    cluster_sync();
    for (int p = 0; p < rank; ++p) {
      const uint2 v = peer_load2(totals, p);
      over0 += v.x;
      tie0 += v.y;
    }
  }
  Order<kThreads, kRounds> order{order_sh};
  for (int r0 = c0; r0 < c1; r0 += kRounds * kThreads) {
    if (r0 > c0) {
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const int at = r0 + i * kThreads + tid;
        x[i] = at < c1 ? w[at] : 0.f;
      }
    }
    auto there = [&](int i) { return r0 + i * kThreads + tid < c1; };
    auto over = [&](int i) { return there(i) && kth.under(ordered(x[i])); };
    auto tie = [&](int i) { return there(i) && kth.holds(ordered(x[i])); };
    const unsigned total = order.scan(over, tie);
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const bool o = over(i), t = tie(i);
      const unsigned before = order.before(i, o, t);
      const int ties = static_cast<int>(tie0 + (before >> 16));
      const int at = static_cast<int>(over0 + (before & 0xffffu)) + min(ties, kth.need);
      if ((o || (t && ties < kth.need)) && at < k) {  // at < k: always, while nobody writes the weights
        kept[at] = r0 + i * kThreads + tid;
        left[at] = x[i];
      }
    }
    over0 += total & 0xffffu;
    tie0 += total >> 16;
    __syncthreads();  // the counts have been read
  }
  if constexpr (kCluster) cluster_sync();  // nobody leaves while others read its shared memory
}

// ---- eviction: the copies
// D / 8 lanes a row, so that a warp copies the keys and values of 32 / (D / 8) kept keys at a time,
// four times ahead.  Bound by reading and writing them once.
constexpr int kMoveThreads = 128, kMoveKeys = 64;  // of a CTA

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, int chunks) {
  constexpr int L = D / 8, kRows = kMoveThreads / L, kSteps = kMoveKeys / kRows;
  begin_launch();
  const CacheSeqs& c = a.c;
  const int bh = static_cast<int>(blockIdx.x) / chunks, chunk = static_cast<int>(blockIdx.x) % chunks;
  const int b = bh / c.Hkv, hk = bh - b * c.Hkv;
  const int sub = threadIdx.x % L, r = threadIdx.x / L;
  const int32_t* kept = a.kept + static_cast<int64_t>(bh) * a.budget;
  const int in_page = (1 << c.page_shift) - 1;
  int64_t from[kSteps], to[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int at = chunk * kMoveKeys + i * kRows + r;
    const int key = at < a.budget ? kept[at] : -1;
    from[i] = to[i] = -1;
    if (key < 0) continue;
    const int src = page_of(c, b, key >> c.page_shift);
    const int dst = resolve_page(a.new_table + static_cast<int64_t>(b) * a.new_pages, a.new_pages, c.num_pages,
                                 c.page_shift, at);
    if (dst < 0) {
      atomicCAS(c.status, 0, kErrIndex);
      continue;
    }
    if (src >= 0)
      from[i] = (((static_cast<int64_t>(src) * c.Hkv + hk) << c.page_shift) + (key & in_page)) * D + sub * 8;
    to[i] = (((static_cast<int64_t>(dst) * c.Hkv + hk) << c.page_shift) + (at & in_page)) * D + sub * 8;
  }
  uint4 kv[2][kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    kv[0][i] = kv[1][i] = make_uint4(0u, 0u, 0u, 0u);  // of a page outside the pool
    if (from[i] >= 0) {
      kv[0][i] = *reinterpret_cast<const uint4*>(a.k_cache + from[i]);
      kv[1][i] = *reinterpret_cast<const uint4*>(a.v_cache + from[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
    if (to[i] >= 0) {
      *reinterpret_cast<uint4*>(a.k_cache + to[i]) = kv[0][i];
      *reinterpret_cast<uint4*>(a.v_cache + to[i]) = kv[1][i];
    }
}

}  // namespace

cudaError_t launch_kv_weights(int d, const WeightsArgs& a, cudaStream_t s) {
  constexpr int kCta = kWeightWarps * kWeightKeys;
  const int chunks = (a.cap + kCta - 1) / kCta;
  const unsigned grid = static_cast<unsigned>(a.c.B) * static_cast<unsigned>(a.c.Hkv) * static_cast<unsigned>(chunks);
  return d == 64 ? launch_chained(kv_weights_kernel<64>, grid, 32 * kWeightWarps, 0, s, a, chunks)
                 : launch_chained(kv_weights_kernel<128>, grid, 32 * kWeightWarps, 0, s, a, chunks);
}

cudaError_t launch_kv_evict(int d, const EvictArgs& a, cudaStream_t s) {
  const unsigned rows = static_cast<unsigned>(a.c.B) * static_cast<unsigned>(a.c.Hkv);
  const int most = a.c.max_len;
  const int cluster = evict_cluster(most, 1024);
  const cudaError_t e =
      most <= kRounds * 256 ? launch_chained(evict_select_kernel<256, false>, rows, 256, 0, s, a)
      : cluster == 1 ? launch_chained(evict_select_kernel<1024, false>, rows, 1024, 0, s, a)
                     : launch_clusters(evict_select_kernel<1024, true>, rows * cluster, cluster, 1024, s, a);
  if (e != cudaSuccess) return e;
  const int chunks = (a.budget + kMoveKeys - 1) / kMoveKeys;
  return d == 64 ? launch_chained(evict_move_kernel<64>, rows * chunks, kMoveThreads, 0, s, a, chunks)
                 : launch_chained(evict_move_kernel<128>, rows * chunks, kMoveThreads, 0, s, a, chunks);
}

}  // namespace fa
