// C-ABI entry points (declared in include/fa.h) of the operators that choose and drop keys of the
// paged cache, and of the mask of a tree.  Every argument is checked before the first launch;
// nothing here allocates device memory.
#include <cmath>

#include "fa.h"
#include "fa_cache.h"
#include "fa_host.h"
#include "serving_checks.h"

namespace {

using fa::aligned_to;
using fa::check_cache;
using fa::check_heads;
using fa::device_ready;
using fa::kMaxInt;
using fa::kMaxKeys;
using fa::page_shift;
using fa::status_of;

constexpr float kLog2e = 1.4426950408889634f;

// Sequences and tokens: B >= 1 sequences, `total` tokens (without offsets, one each).
fa_status check_tokens(int B, int total, const int32_t* cu) {
  if (B < 1 || B > (1 << 29) || total < 0) return FA_ERR_INVALID_ARG;
  return cu == nullptr && total != B ? FA_ERR_INVALID_ARG : FA_OK;
}

fa::CacheSeqs seqs_of(const fa_paged_kv& c, const int32_t* cu, int B, int total, int max_kv, int Hkv,
                      int* status) {
  fa::CacheSeqs s{};
  s.block_table = c.block_table;
  s.kv_lens = c.kv_lens;
  s.cu = cu;
  s.B = B;
  s.total = total;
  s.max_pages = c.max_pages;
  s.num_pages = c.num_pages;
  s.page_shift = page_shift(c.page_size);
  s.max_len = max_kv < kMaxKeys ? max_kv : kMaxKeys;
  s.Hkv = Hkv;
  s.status = status;
  return s;
}

// Pages of a sequence of max_kv keys.
long long pages_of(int max_kv, int page_size) {
  const long long keys = max_kv < kMaxKeys ? max_kv : kMaxKeys;
  return (keys + page_size - 1) / page_size;
}

// Work items of a launch, or of one of its arrays' rows, that fit 31 bits.
bool fits(long long a, long long b, long long c) {
  return a * b <= kMaxInt && a * b * c <= kMaxInt;
}

}  // namespace

extern "C" {

fa_status fa_tree_mask(const int32_t* parents, const int32_t* cu_seqlens, int B, int total,
                       int mask_words, uint64_t* tree_mask, void* stream) {
  fa_status st = check_tokens(B, total, cu_seqlens);
  if (st != FA_OK) return st;
  if (mask_words < 1 || mask_words > (1 << 24)) return FA_ERR_INVALID_ARG;
  if (total == 0) return FA_OK;
  if (!parents || !tree_mask || !aligned_to(parents, 4) || !aligned_to(tree_mask, 8))
    return FA_ERR_INVALID_ARG;
  int* status = nullptr;
  if ((st = device_ready(status)) != FA_OK) return st;
  return status_of(fa::launch_tree_mask(parents, cu_seqlens, B, total, mask_words, tree_mask, status,
                                        static_cast<cudaStream_t>(stream)));
}

fa_status fa_page_bounds(const fa_paged_kv* cache, void* bounds, const int32_t* cu_seqlens, int B,
                         int total, int Hkv, int d, void* stream) {
  fa_status st = check_heads(Hkv, Hkv, d);
  if (st != FA_OK) return st;
  if ((st = check_cache(cache, true, false)) != FA_OK) return st;
  if ((st = check_tokens(B, total, cu_seqlens)) != FA_OK) return st;
  if (!bounds || !aligned_to(bounds, 16)) return FA_ERR_INVALID_ARG;
  if (!fits(total / cache->page_size + 2LL * B, Hkv, 1)) return FA_ERR_UNSUPPORTED;
  if (total == 0) return FA_OK;
  fa::BoundsArgs a{};
  int* status = nullptr;
  if ((st = device_ready(status)) != FA_OK) return st;
  a.c = seqs_of(*cache, cu_seqlens, B, total, kMaxInt, Hkv, status);
  a.k_cache = static_cast<const __nv_bfloat16*>(cache->k_cache);
  a.bounds = static_cast<__nv_bfloat16*>(bounds);
  return status_of(fa::launch_page_bounds(d, a, static_cast<cudaStream_t>(stream)));
}

size_t fa_select_pages_workspace_size(int B, int total, int Hkv, int page_size, int max_kv) {
  if (B < 1 || total < 0 || Hkv < 1 || max_kv < 0 || page_shift(page_size) < 0) return 0;
  return fa::select_workspace(B, total, Hkv, static_cast<int>(pages_of(max_kv, page_size))).total;
}

fa_status fa_select_pages(const void* Q, const void* bounds, const fa_paged_kv* cache,
                          int32_t* pages, int top, int first, int last, const int32_t* cu_seqlens,
                          int B, int max_kv, int total, int H, int Hkv, int d, void* workspace,
                          size_t workspace_bytes, void* stream) {
  fa_status st = check_heads(H, Hkv, d);
  if (st != FA_OK) return st;
  if (H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (H / Hkv > 128) return FA_ERR_UNSUPPORTED;
  if ((st = check_cache(cache, false, false)) != FA_OK) return st;
  if ((st = check_tokens(B, total, cu_seqlens)) != FA_OK) return st;
  if (top < 1 || first < 0 || last < 0 || first > top || last > top - first || max_kv < 0)
    return FA_ERR_INVALID_ARG;
  if (total == 0) return FA_OK;
  if (!Q || !bounds || !pages || !aligned_to(Q, 16) || !aligned_to(bounds, 16))
    return FA_ERR_INVALID_ARG;
  const long long most = pages_of(max_kv, cache->page_size);
  if (!fits(B, Hkv, most / 32 + 1) || !fits(total, Hkv, 1)) return FA_ERR_UNSUPPORTED;
  const fa::SelectWorkspace w = fa::select_workspace(B, total, Hkv, static_cast<int>(most));
  if ((st = fa::check_workspace(workspace, workspace_bytes, w.total)) != FA_OK) return st;
  fa::SelectArgs a{};
  int* status = nullptr;
  if ((st = device_ready(status)) != FA_OK) return st;
  a.c = seqs_of(*cache, cu_seqlens, B, total, max_kv, Hkv, status);
  a.q = static_cast<const __nv_bfloat16*>(Q);
  a.bounds = static_cast<const __nv_bfloat16*>(bounds);
  a.H = H;
  a.G = H / Hkv;
  a.max_pages = static_cast<int>(most);
  a.top = top;
  a.first = first;
  a.last = last;
  a.pages = pages;
  char* base = static_cast<char*>(workspace);
  a.score = reinterpret_cast<float*>(base + w.score);
  a.fine = reinterpret_cast<uint64_t*>(base + w.fine);
  a.reach = reinterpret_cast<float*>(base + w.reach);
  return status_of(fa::launch_select_pages(d, a, static_cast<cudaStream_t>(stream)));
}

fa_status fa_kv_weights(const void* Q, const float* LSE, const fa_paged_kv* cache,
                        const float* weights, float* out, int capacity, const int32_t* cu_seqlens,
                        int B, int max_q, int max_kv, int total, int H, int Hkv, int d, int causal,
                        float scale, void* stream) {
  fa_status st = check_heads(H, Hkv, d);
  if (st != FA_OK) return st;
  if (H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (H / Hkv > 128) return FA_ERR_UNSUPPORTED;
  if ((st = check_cache(cache, true, false)) != FA_OK) return st;
  if ((st = check_tokens(B, total, cu_seqlens)) != FA_OK) return st;
  if (max_q < 1 || max_kv < 0 || capacity < 0 || capacity > kMaxKeys || !std::isfinite(scale))
    return FA_ERR_INVALID_ARG;
  if (capacity == 0) return FA_OK;
  if (!out || (total > 0 && (!Q || !LSE || !aligned_to(Q, 16)))) return FA_ERR_INVALID_ARG;
  // the index of a (token, head) row, and the units of the launch
  const int len = max_kv < capacity ? max_kv : capacity;
  if (!fits(total, H, 1) || static_cast<long long>(total) * (H / Hkv) > fa::kWeightsRows ||
      !fits(B, Hkv, len / 128 + 3) || static_cast<long long>(cache->num_pages) * Hkv > kMaxInt)
    return FA_ERR_UNSUPPORTED;
  fa::PagedArgs a{};
  if ((st = device_ready(a.status)) != FA_OK) return st;
  CUtensorMap tk;
  if (!fa::make_pool_map(&tk, cache->k_cache, *cache, Hkv, d)) return FA_ERR_CUDA;
  a.q = static_cast<const __nv_bfloat16*>(Q);
  a.cu = cu_seqlens;
  a.B = B;
  a.total = total;
  a.H = H;
  a.Hkv = Hkv;
  a.G = H / Hkv;
  a.num_pages = cache->num_pages;
  a.page_shift = page_shift(cache->page_size);
  a.scale_log2 = fa::resolve_scale(scale, d) * kLog2e;
  fa::KeyList& l = a.list[0];
  l.count = B;
  l.lens = cache->kv_lens;
  l.table = cache->block_table;
  l.max_pages = cache->max_pages;
  l.max_len = len;
  l.max_q = max_q;
  // (one token of 64 sequences of 512 to 4096 keys: 56.8 us, with 0 58.8; 256 such sequences 206 and 211;
  // the CTAs' times fit 0.9 to 1.1 tiles a segment at 4 queries and 2.2 at 128)
  l.extra = static_cast<long long>(total) * a.G >= 64LL * B ? 2 : 1;
  const fa::WeightsOut w{LSE, weights, out, capacity, causal != 0};
  return status_of(fa::launch_kv_weights(d, tk, a, w, fa::wait_timeout_ns(), static_cast<cudaStream_t>(stream)));
}

fa_status fa_kv_evict(const float* weights, int capacity, const fa_paged_kv* cache,
                      const int32_t* new_table, int new_pages, int budget, int recent,
                      int32_t* new_lens, int32_t* kept, float* new_weights, int B, int max_kv,
                      int Hkv, int d, void* stream) {
  fa_status st = check_heads(Hkv, Hkv, d);
  if (st != FA_OK) return st;
  if ((st = check_cache(cache)) != FA_OK) return st;
  if (B < 1 || B > (1 << 29) || max_kv < 0 || capacity < 0 || capacity > kMaxKeys || budget < 1 ||
      budget > kMaxKeys || recent < 0 || recent > budget || new_pages < 0)
    return FA_ERR_INVALID_ARG;
  if ((capacity > 0 && !weights) || (new_pages > 0 && !new_table) || !new_lens || !kept || !new_weights)
    return FA_ERR_INVALID_ARG;
  if (!fits(B, Hkv, budget / 16 + 8)) return FA_ERR_UNSUPPORTED;
  fa::EvictArgs a{};
  int* status = nullptr;
  if ((st = device_ready(status)) != FA_OK) return st;
  a.c = seqs_of(*cache, nullptr, B, B, max_kv < capacity ? max_kv : capacity, Hkv, status);
  a.weights = weights;
  a.cap = capacity;
  a.budget = budget;
  a.recent = recent;
  a.k_cache = static_cast<__nv_bfloat16*>(cache->k_cache);
  a.v_cache = static_cast<__nv_bfloat16*>(cache->v_cache);
  a.new_table = new_table;
  a.new_pages = new_pages;
  a.new_lens = new_lens;
  a.kept = kept;
  a.new_weights = new_weights;
  return status_of(fa::launch_kv_evict(d, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
