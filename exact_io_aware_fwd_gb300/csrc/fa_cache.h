// Internal interface of the operators that choose and drop keys of the paged cache: the bounds of
// pages and the selection of pages for each query (fa_pages.cu), accumulated attention weights
// (fa_weights.cu) and eviction (fa_evict.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_paged.h"

namespace fa {

// Sequences of the paged cache and their new tokens.
struct CacheSeqs {
  const int32_t *block_table, *kv_lens, *cu;
  int B, total, max_pages, num_pages, page_shift;
  int max_len;  // lengths are clamped to it
  int Hkv;
  int* status;
};

// Pages that hold one of the last n keys of a sequence are at most n / page_size + 2, so slot
// cu[b] / page_size + 2 b + i stands for the i-th of sequence b: disjoint, whatever the lengths.
__host__ __device__ __forceinline__ int first_slot(const int32_t* cu, int b, int total, int shift) {
#ifdef __CUDA_ARCH__
  const int at = cu != nullptr ? __ldg(cu + b) : b;
#else
  const int at = cu != nullptr ? cu[b] : b;
#endif
  return (min(max(at, 0), total) >> shift) + 2 * b;
}

// Whether offsets [t0, t1) of a sequence of `len` keys leave its pages out: they are none, or `total`
// cuts new tokens off whose pages its other ones do not lie in.
__host__ __device__ inline bool pages_left_out(int t0, int t1, int total, int len, int shift) {
  if (t0 < 0 || t1 < t0) return true;
  int start, n;
  clamp_tokens(t0, t1, total, start, n);
  if (n == t1 - t0 || len == 0) return false;
  const int all = t1 - t0 < len ? len - (t1 - t0) : 0, some = n < len ? len - n : 0;
  return n == 0 || some >> shift > all >> shift;
}

#ifdef __CUDACC__
// Keys of sequence b, clamped (and reported).
__device__ __forceinline__ int keys_of(const CacheSeqs& c, int b, bool report) {
  const int len = __ldg(c.kv_lens + b);
  const int64_t reach = static_cast<int64_t>(c.max_pages) << c.page_shift;
  const int cap = reach < c.max_len ? static_cast<int>(reach) : c.max_len;
  const int n = min(max(len, 0), cap);
  if (report && n != len) atomicCAS(c.status, 0, kErrIndex);
  return n;
}
// Page number `i` of sequence b, or -1 (reported) outside the pool.
__device__ __forceinline__ int page_of(const CacheSeqs& c, int b, int i) {
  const int p = resolve_page(c.block_table + static_cast<int64_t>(b) * c.max_pages, c.max_pages,
                             c.num_pages, c.page_shift, i << c.page_shift);
  if (p < 0) atomicCAS(c.status, 0, kErrIndex);
  return p;
}
// A float's bits in the order of the numbers: -0 as 0, NaN above infinity.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t ordered(double x) {
  if (x != x) return ~0ull;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return u >> 63 ? ~u : u | (1ull << 63);
}
#endif

// Ancestors of the tokens of trees (fa_pages.cu).
cudaError_t launch_tree_mask(const int32_t* parents, const int32_t* cu, int B, int total, int words,
                             uint64_t* mask, int* status, cudaStream_t s);

// ---- bounds of pages and their selection (fa_pages.cu)
struct BoundsArgs {
  CacheSeqs c;
  const __nv_bfloat16* k_cache;
  __nv_bfloat16* bounds;  // [num_pages][Hkv][2][d]
};
cudaError_t launch_page_bounds(int d, const BoundsArgs& a, cudaStream_t s);

struct SelectArgs {
  CacheSeqs c;
  const __nv_bfloat16 *q, *bounds;
  int H, G;
  int max_pages;      // of a sequence, by max_len
  int top, first, last;
  int32_t* pages;     // [total][Hkv][top]
  float* score;       // workspace: [total][Hkv][max_pages]
  uint64_t* fine;     // workspace: the same exactly, where many scores are next to the border
  float* reach;       // workspace: [B][Hkv][ceil(max_pages / 16)] largest |bound| of 16 pages
};
struct SelectWorkspace {
  size_t score, fine, reach, total;
};
SelectWorkspace select_workspace(int B, int total, int Hkv, int max_pages);
cudaError_t launch_select_pages(int d, const SelectArgs& a, cudaStream_t s);

// ---- accumulated weights (fa_weights.cu): the sequences and queries are those of a PagedArgs with
// one list, whose causal is 0 (every key is visited)
struct WeightsOut {
  const float *lse, *in;  // in: nullptr or [B][Hkv][cap]
  float* out;             // [B][Hkv][cap]
  int cap, causal;
};
constexpr long long kWeightsRows = 1 << 29;  // queries of a launch for a key/value head
cudaError_t launch_kv_weights(int d, const CUtensorMap& tk, const PagedArgs& a, const WeightsOut& w,
                              uint64_t timeout_ns, cudaStream_t s);

// ---- eviction (fa_evict.cu)
struct EvictArgs {
  CacheSeqs c;
  const float* weights;   // [B][Hkv][cap]
  int cap, budget, recent;
  __nv_bfloat16 *k_cache, *v_cache;
  const int32_t* new_table;  // [B][new_pages]
  int new_pages;
  int32_t *new_lens, *kept;  // [B], [B][Hkv][budget]
  float* new_weights;        // [B][Hkv][budget]
};
cudaError_t launch_kv_evict(int d, const EvictArgs& a, cudaStream_t s);

}  // namespace fa
