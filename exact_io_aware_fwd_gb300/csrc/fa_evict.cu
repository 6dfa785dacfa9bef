// Eviction of the keys that have gathered the least attention.
#include "fa_cache.h"
#include "fa_internal.h"
#include "select_kth.cuh"
#include "sm103.cuh"

namespace fa {

namespace {

// ---- eviction: which keys stay
// The smallest weight that stays by counting (select_kth.cuh), then the keys in order.  A sequence
// and head is a CTA's, or, where a CTA's registers (kRounds weights a thread) do not hold its
// weights, a cluster's, each CTA with a stretch of them; only what does not fit eight CTAs is read
// again in every pass.
// Clusters of more than eight CTAs do not all run at once (the selection of 8 heads of 131072 keys, cold:
// 16 of 512 threads 37 us, 8 of 1024 20).
constexpr int kRounds = 8, kMoreRounds = 16;
constexpr int evict_cluster(int max_len, int threads) {
  int c = 2;
  while (c < static_cast<int>(kMostPeers) && c * kMoreRounds * threads < max_len) c *= 2;
  return c;
}

template <int kThreads, int kRounds, bool kCluster>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictArgs a) {
  constexpr int kHeld = kRounds * kThreads;
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
  // this CTA's stretch; what its registers hold, as numbers that order like the weights
  const int chunk = (old + ctas - 1) / ctas, c0 = min(old, rank * chunk), c1 = min(old, c0 + chunk);
  // (0, which no weight gives, where there is none).  All loads are on the way before the first is
  // used.
  uint32_t x[kRounds];
  auto read = [&](int r0) {
    float v[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) v[i] = w[max(min(r0 + i * kThreads + tid, c1 - 1), 0)];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) asm volatile("" : "+f"(v[i]));
#pragma unroll
    for (int i = 0; i < kRounds; ++i) x[i] = r0 + i * kThreads + tid < c1 ? ordered(v[i]) : 0u;
  };
  if (k > 0) read(c0);
  for (int i = count + all; i < a.budget; i += ctas * kThreads) {
    kept[i] = -1;
    left[i] = 0.f;
  }
  for (int i = old + all; i < len; i += ctas * kThreads) {
    kept[k + i - old] = i;
    left[k + i - old] = w[i];
  }
  if (k == 0) return;  // the whole cluster
  auto tail = [&](auto f) {
    for (int at = c0 + kHeld + tid; at < c1; at += kThreads) f(ordered(w[at]));
  };
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      if (x[i] != 0u) f(x[i]);
    tail(f);
  };
  const Kth<uint32_t> kth = kth_largest<kThreads, kCluster, uint32_t>(k, 0, each, sh);
  Order<kThreads, kRounds> order{order_sh};
  unsigned over0 = 0, tie0 = 0;  // in front of what comes next
  for (int r0 = c0; r0 == c0 || r0 < c1; r0 += kHeld) {
    if (r0 > c0) read(r0);
    const unsigned total = order.scan([&](int i) { return kth.under(x[i]); }, [&](int i) { return kth.holds(x[i]); });
    if constexpr (kCluster) {
      if (r0 == c0) {  // what the CTAs in front have
        if (tid == 0) {
          totals[0] = total & 0xffffu;
          totals[1] = total >> 16;
        }
        __syncthreads();
        if (c1 - c0 > kHeld) {
          unsigned over = 0, tie = 0;
          tail([&](uint32_t key) {
            over += kth.under(key);
            tie += kth.holds(key);
          });
          over = __reduce_add_sync(~0u, over);
          tie = __reduce_add_sync(~0u, tie);
          if ((tid & 31) == 0) {
            atomicAdd(&totals[0], over);
            atomicAdd(&totals[1], tie);
          }
        }
        cluster_sync();
        const int p = tid & 31;
        const uint2 v = p < rank ? peer_load2(totals, p) : make_uint2(0u, 0u);
        over0 = __reduce_add_sync(~0u, v.x);
        tie0 = __reduce_add_sync(~0u, v.y);
        cluster_arrive();  // nothing of another CTA's is read any more
      }
    }
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const unsigned before = order.before(i);
      const int ties = static_cast<int>(tie0 + (before >> 16));
      const int at = static_cast<int>(over0 + (before & 0xffffu)) + min(ties, kth.need);
      // at < k: always, while nobody writes the weights
      if ((order.over(i) || (order.tie(i) && ties < kth.need)) && at < k) {
        kept[at] = r0 + i * kThreads + tid;
        left[at] = unordered(x[i]);
      }
    }
    over0 += total & 0xffffu;
    tie0 += total >> 16;
    __syncthreads();  // the counts have been read
  }
  if constexpr (kCluster) cluster_wait();  // nobody leaves while others read its shared memory
}

// ---- eviction: the copies
// D / 8 lanes a row, the keys and values of two kept keys a thread on the way.  Bound by reading and
// writing them once.  Neither is read again soon, so neither stays in L2 (90.6 us for 64 sequences of
// 512 to 4096 keys to 1024; stores that stay 93.8, both 91.8); eight keys a thread, in flight just as
// long but fewer at a time near the end: 105.
constexpr int kMoveThreads = 128, kMoveSteps = 2;
__host__ __device__ constexpr int move_keys(int d) { return kMoveSteps * kMoveThreads * 8 / d; }  // of a CTA

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, int chunks) {
  constexpr int L = D / 8, kRows = kMoveThreads / L, kSteps = kMoveSteps, kMoveKeys = move_keys(D);
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
      kv[0][i] = __ldcs(reinterpret_cast<const uint4*>(a.k_cache + from[i]));
      kv[1][i] = __ldcs(reinterpret_cast<const uint4*>(a.v_cache + from[i]));
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
    if (to[i] >= 0) {
      __stcs(reinterpret_cast<uint4*>(a.k_cache + to[i]), kv[0][i]);
      __stcs(reinterpret_cast<uint4*>(a.v_cache + to[i]), kv[1][i]);
    }
}

}  // namespace

cudaError_t launch_kv_evict(int d, const EvictArgs& a, cudaStream_t s) {
  const unsigned rows = static_cast<unsigned>(a.c.B) * static_cast<unsigned>(a.c.Hkv);
  const int most = a.c.max_len;
  cudaError_t e;
  if (most <= kRounds * 256) {
    e = launch_chained(evict_select_kernel<256, kRounds, false>, rows, 256, 0, s, a);
  } else if (most <= kMoreRounds * 256) {
    e = launch_chained(evict_select_kernel<256, kMoreRounds, false>, rows, 256, 0, s, a);
  } else if (most <= kRounds * 1024) {
    e = launch_chained(evict_select_kernel<1024, kRounds, false>, rows, 1024, 0, s, a);
  } else if (most <= static_cast<int>(kMostPeers) * kMoreRounds * 512) {
    const int c = evict_cluster(most, 512);
    e = launch_clusters(evict_select_kernel<512, kMoreRounds, true>, rows * c, c, 512, s, a);
  } else {
    const int c = evict_cluster(most, 1024);
    e = launch_clusters(evict_select_kernel<1024, kMoreRounds, true>, rows * c, c, 1024, s, a);
  }
  if (e != cudaSuccess) return e;
  const int chunks = (a.budget + move_keys(d) - 1) / move_keys(d);
  return d == 64 ? launch_chained(evict_move_kernel<64>, rows * chunks, kMoveThreads, 0, s, a, chunks)
                 : launch_chained(evict_move_kernel<128>, rows * chunks, kMoveThreads, 0, s, a, chunks);
}

}  // namespace fa
