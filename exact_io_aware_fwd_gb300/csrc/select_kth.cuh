// The k-th largest of many keys held by a CTA or by the CTAs of a cluster, by counting, and the order
// in which what was selected is listed.
//
// Each pass sorts the keys that are still in question into 2048 equal bins and goes on with the bin
// that holds the k-th.  The bins divide the range that the keys really have, so the first pass spreads
// them (the leading bits of floats that lie close together are the same) and rarely more than two
// passes are needed.  A cluster's CTAs add up each other's bins through distributed shared memory,
// one cluster barrier a pass; each of them reads all bins of all, so a cluster has 1024 (eviction of
// 131072 keys: 36.9 us, with 2048 37.7; of eight such sequences 246 us, 257).
#pragma once

#include <cstdint>

#include "sm103.cuh"

namespace fa {

// ---- the CTAs of a cluster
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of all its CTAs.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// Shared-memory words of CTA `rank`, at the address that `p` has here.
__device__ __forceinline__ uint32_t peer_load(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
      "ld.shared::cluster.u32 %0, [a];\n\t}"
      : "=r"(v)
      : "r"(smem_u32(p)), "r"(rank)
      : "memory");
  return v;
}
__device__ __forceinline__ uint2 peer_load2(const void* p, uint32_t rank) {
  uint2 v;
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\t"
      "ld.shared::cluster.v2.u32 {%0, %1}, [a];\n\t}"
      : "=r"(v.x), "=r"(v.y)
      : "r"(smem_u32(p)), "r"(rank)
      : "memory");
  return v;
}

// Over a warp's lanes.
__device__ __forceinline__ uint32_t lanes_min(uint32_t x) { return __reduce_min_sync(~0u, x); }
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) { return __reduce_max_sync(~0u, x); }
__device__ __forceinline__ uint64_t lanes_min(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t y = __shfl_xor_sync(~0u, x, o);
    x = y < x ? y : x;
  }
  return x;
}
__device__ __forceinline__ uint64_t lanes_max(uint64_t x) { return ~lanes_min(~x); }
// Of the warps' values (one each, in shared memory): the sum, and that of the warps before this one.
template <int kWarps>
__device__ __forceinline__ unsigned sum_of(const unsigned* v) {
  const int lane = threadIdx.x & 31;
  return __reduce_add_sync(~0u, lane < kWarps ? v[lane] : 0u);
}
template <int kWarps>
__device__ __forceinline__ unsigned sum_before(const unsigned* v) {
  const int lane = threadIdx.x & 31;
  return __reduce_add_sync(~0u, lane < static_cast<int>(threadIdx.x >> 5) ? v[lane] : 0u);
}

constexpr int kKthBins = 2048, kClusterBins = 1024;
constexpr uint32_t kMostPeers = 8;  // CTAs of a cluster

template <int kThreads, typename Key>
struct KthShared {
  alignas(8) unsigned hist[2][kKthBins];
  alignas(8) Key lo[kThreads / 32], hi[kThreads / 32];  // of the warps; [0]: then of the CTA
  alignas(8) Key ends[2];                               // smallest and largest of the CTA
  unsigned warp_sum[kThreads / 32];
  int bin, need, count;
};

// The k-th largest key lies in [base, base + range]; `need` of the `count` keys in there belong to
// the k largest, and every key above does.
template <typename Key>
struct Kth {
  Key base, range;
  int need, count;
  __device__ bool holds(Key key) const { return key - base <= range; }  // (a smaller key wraps)
  __device__ bool under(Key key) const { return key > base + range; }
};

__device__ __forceinline__ int bit_length(uint32_t x) { return 32 - __clz(x); }
__device__ __forceinline__ int bit_length(uint64_t x) { return 64 - __clzll(x); }

// each(f) calls f(key) for every key of this thread.  1 <= k <= number of keys.  Ends when every key
// of the range is needed, when the range is one key, or when it holds no more than `few` keys.  Called
// by all threads of the CTA, or (kCluster, 32-bit keys) of the cluster; sh may be used again after the
// next barrier.
template <int kThreads, bool kCluster, typename Key, typename Each>
__device__ __forceinline__ Kth<Key> kth_largest(int k, int few, Each each,
                                                KthShared<kThreads, Key>& sh) {
  static_assert(!kCluster || sizeof(Key) == 4, "peers' ends are read as a pair of words");
  constexpr int kBins = kCluster ? kClusterBins : kKthBins, kBits = kBins == 2048 ? 11 : 10;
  constexpr int kWarps = kThreads / 32, kOwn = kBins / kThreads;
  static_assert(kOwn * kThreads == kBins && 1 << kBits == kBins, "bins per thread");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t peers = kCluster ? cluster_size() : 1;
  Key lo = ~Key(0), hi = 0;
  each([&](Key key) {
    lo = key < lo ? key : lo;
    hi = key > hi ? key : hi;
  });
  lo = lanes_min(lo);
  hi = lanes_max(hi);
  if (lane == 0) {
    sh.lo[warp] = lo;
    sh.hi[warp] = hi;
  }
#pragma unroll
  for (int i = 0; i < kOwn; ++i) sh.hist[0][i * kThreads + tid] = sh.hist[1][i * kThreads + tid] = 0;
  __syncthreads();
  lo = lanes_min(lane < kWarps ? sh.lo[lane] : ~Key(0));
  hi = lanes_max(lane < kWarps ? sh.hi[lane] : Key(0));
  if constexpr (kCluster) {
    if (tid == 0) {
      sh.ends[0] = lo;
      sh.ends[1] = hi;
    }
    cluster_sync();
    const uint2 v = peer_load2(&sh.ends[0], min(static_cast<uint32_t>(lane), peers - 1));
    lo = __reduce_min_sync(~0u, v.x);
    hi = __reduce_max_sync(~0u, v.y);
  }
  Kth<Key> r{lo, hi - lo, k, -1};
  for (int pass = 0;; ++pass) {  // a pass leaves at most a 1024th of the range (clusters: a 512th)
    const int bits = bit_length(r.range), shift = bits > kBits ? bits - kBits : 0;
    // two sets of bins take turns: this one is empty, and the other is cleared once nobody reads it
    unsigned* const hist = sh.hist[pass & 1];
    if (pass == 0) {
      each([&](Key key) { atomicAdd(&hist[static_cast<unsigned>((key - r.base) >> shift)], 1u); });
    } else {
      each([&](Key key) {
        if (r.holds(key)) atomicAdd(&hist[static_cast<unsigned>((key - r.base) >> shift)], 1u);
      });
    }
    if constexpr (kCluster) cluster_sync();
    else __syncthreads();
    // thread t owns the kOwn bins from own0 down, counted from the top
    unsigned mine[kOwn], sum = 0;
    const int own0 = kBins - 1 - tid * kOwn;
    if constexpr (kCluster) {
      unsigned v[kMostPeers][kOwn];  // on the way together
#pragma unroll
      for (uint32_t p = 0; p < kMostPeers; ++p)
#pragma unroll
        for (int i = 0; i < kOwn; ++i) v[p][i] = p < peers ? peer_load(&hist[own0 - i], p) : 0u;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        mine[i] = 0;
#pragma unroll
        for (uint32_t p = 0; p < kMostPeers; ++p) mine[i] += v[p][i];
      }
    } else {
      static_assert(kOwn % 2 == 0 || kCluster, "bins are read in pairs");
#pragma unroll
      for (int i = 0; i < kOwn; i += 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(&hist[own0 - i - 1]);
        mine[i] = v.y;
        mine[i + 1] = v.x;
      }
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) sum += mine[i];
    unsigned incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    unsigned above = incl - sum + sum_before<kWarps>(sh.warp_sum);
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const unsigned need = static_cast<unsigned>(r.need);
      if (above < need && need <= above + mine[i]) {
        sh.bin = own0 - i;
        sh.need = static_cast<int>(need - above);
        sh.count = static_cast<int>(mine[i]);
      }
      above += mine[i];
    }
    if (pass > 0) {  // read by others before this pass' barrier; filled after the next one
#pragma unroll
      for (int i = 0; i < kOwn; ++i) sh.hist[(pass & 1) ^ 1][i * kThreads + tid] = 0;
    }
    __syncthreads();
    const Key step = static_cast<Key>(sh.bin) << shift;
    r.base += step;
    const Key left = r.range - step, width = (Key(1) << shift) - 1;
    r.range = left < width ? left : width;
    r.need = sh.need;
    r.count = sh.count;
    if (shift == 0 || r.need == r.count || r.count <= few) break;  // the same everywhere
  }
  return r;
}

// Places in order: element (i, thread) of a CTA's kRounds x kThreads elements, rounds first, has
// `over` elements above the k-th and `tie` ones in its range in front of it.
template <int kThreads, int kRounds>
struct OrderShared {
  unsigned count[kRounds * kThreads / 32];  // over, tie << 16 of each round and warp
  unsigned warp_sum[kThreads / 32];
};
template <int kThreads, int kRounds>
struct Order {
  static constexpr int kWarps = kThreads / 32, kEntries = kRounds * kWarps;
  static_assert(kEntries <= kThreads && kRounds * kThreads < 65536, "a thread an entry, 16 bits a count");
  OrderShared<kThreads, kRounds>& sh;

  unsigned o[kRounds], t[kRounds];  // the warp's votes

  // over(i), tie(i): of this thread's element of round i.  Returns the totals (tie << 16).
  template <typename Over, typename Tie>
  __device__ __forceinline__ unsigned scan(Over over, Tie tie) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      o[i] = __ballot_sync(~0u, over(i));
      t[i] = __ballot_sync(~0u, tie(i));
      if (lane == 0) sh.count[i * kWarps + warp] = __popc(o[i]) | __popc(t[i]) << 16;
    }
    __syncthreads();
    const unsigned own = tid < kEntries ? sh.count[tid] : 0u;
    unsigned incl = own;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const unsigned v = __shfl_up_sync(~0u, incl, x);
      if (lane >= x) incl += v;
    }
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    incl += sum_before<kWarps>(sh.warp_sum);
    const unsigned total = sum_of<kWarps>(sh.warp_sum);
    if (tid < kEntries) sh.count[tid] = incl - own;
    __syncthreads();
    return total;
  }
  // Whether this thread's element of round i was one, and (over, tie << 16) in front of it.
  __device__ __forceinline__ bool over(int i) const { return o[i] >> (threadIdx.x & 31) & 1u; }
  __device__ __forceinline__ bool tie(int i) const { return t[i] >> (threadIdx.x & 31) & 1u; }
  __device__ __forceinline__ unsigned before(int i) const {
    const unsigned less = (1u << (threadIdx.x & 31)) - 1u;
    return sh.count[i * kWarps + (threadIdx.x >> 5)] + (__popc(o[i] & less) | __popc(t[i] & less) << 16);
  }
};

}  // namespace fa
