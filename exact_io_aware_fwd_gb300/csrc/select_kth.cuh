// The k-th largest of a CTA's keys, by counting: each pass sorts the keys that are still in question
// into 2048 equal bins and goes on with the bin that holds the k-th.  The bins divide the range that
// the keys really have, so the first pass spreads them (the leading bits of floats that lie close
// together are the same) and rarely more than two passes are needed.
#pragma once

#include <cstdint>

namespace fa {

constexpr int kKthBins = 2048;

template <int kThreads, typename Key>
struct KthShared {
  unsigned hist[kKthBins];
  unsigned warp_sum[kThreads / 32];
  Key lo[kThreads / 32], hi[kThreads / 32];
  int bin, need, count;
};

// The k-th largest key lies in [base, base + range]; `need` of the `count` keys in there belong to
// the k largest, and every key above does.
template <typename Key>
struct Kth {
  Key base, range;
  int need, count;
};

__device__ __forceinline__ int bit_length(uint32_t x) { return 32 - __clz(x); }
__device__ __forceinline__ int bit_length(uint64_t x) { return 64 - __clzll(x); }

// load(i, key): whether element i < n counts, and its key.  1 <= k <= number that count.  Ends when
// every key of the range is needed, when the range is one key, or after max_passes.  Called by all
// kThreads threads; sh may be used again after the next barrier.
template <int kThreads, typename Key, typename Load>
__device__ Kth<Key> kth_largest(int n, int k, int max_passes, Load load, KthShared<kThreads, Key>& sh) {
  constexpr int kWarps = kThreads / 32, kOwn = kKthBins / kThreads;
  static_assert(kOwn >= 1 && kOwn * kThreads == kKthBins, "bins per thread");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Key lo = ~Key(0), hi = 0;
  for (int i = tid; i < n; i += kThreads) {
    Key key;
    if (load(i, key)) {
      lo = key < lo ? key : lo;
      hi = key > hi ? key : hi;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Key l = __shfl_xor_sync(~0u, lo, o), h = __shfl_xor_sync(~0u, hi, o);
    lo = l < lo ? l : lo;
    hi = h > hi ? h : hi;
  }
  if (lane == 0) {
    sh.lo[warp] = lo;
    sh.hi[warp] = hi;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    lo = sh.lo[w] < lo ? sh.lo[w] : lo;
    hi = sh.hi[w] > hi ? sh.hi[w] : hi;
  }
  Kth<Key> r{lo, hi - lo, k, -1};
  for (int pass = 0; pass < max_passes; ++pass) {
    const int bits = bit_length(r.range), shift = bits > 11 ? bits - 11 : 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) sh.hist[i * kThreads + tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      Key key;
      if (load(i, key) && key >= r.base && key - r.base <= r.range)
        atomicAdd(&sh.hist[static_cast<unsigned>((key - r.base) >> shift)], 1u);
    }
    __syncthreads();
    // thread t owns the bins [own0, own0 + kOwn), counted from the top
    unsigned mine[kOwn], sum = 0;
    const int own0 = kKthBins - 1 - tid * kOwn;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) sum += mine[i] = sh.hist[own0 - i];
    unsigned incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    unsigned above = incl - sum;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (w < warp) above += sh.warp_sum[w];
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
    __syncthreads();
    const Key step = static_cast<Key>(sh.bin) << shift;
    r.base += step;
    const Key left = r.range - step, width = (Key(1) << shift) - 1;
    r.range = left < width ? left : width;
    r.need = sh.need;
    r.count = sh.count;
    if (shift == 0 || r.need == r.count) break;  // uniform
  }
  return r;
}

}  // namespace fa
