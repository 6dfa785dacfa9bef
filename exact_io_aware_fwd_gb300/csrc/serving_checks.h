// Argument checks that the entry points of the operators around attention share.
#pragma once

#include <atomic>

#include <cuda_runtime.h>

#include "fa.h"
#include "fa_host.h"

namespace fa {

constexpr int kMaxInt = 0x7fffffff;
constexpr int kMaxKeys = kMaxInt - 255;  // keys rounded up to whole tiles fit 32 bits

inline fa_status check_heads(int H, int Hkv, int d) {
  if (H <= 0 || Hkv <= 0) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(H) + 2LL * Hkv > 65535) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// The current device is an sm_103 part (asked once per device); its status word.
inline fa_status device_ready(int*& status) {
  static std::atomic<uint64_t> ready{0};  // bit d: device d is one
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if ((ready.load(std::memory_order_acquire) & bit) == 0) {
    const fa_status st = check_device();
    if (st != FA_OK) return st;
    ready.fetch_or(bit, std::memory_order_release);
  }
  status = status_ptr();
  return status == nullptr ? FA_ERR_CUDA : FA_OK;
}

inline int page_shift(int page_size) {
  switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
  }
  return -1;
}

// keys, values: whether the call reads or writes them.
inline fa_status check_cache(const fa_paged_kv* c, bool keys = true, bool values = true) {
  if (c == nullptr || c->kv_lens == nullptr || (keys && c->k_cache == nullptr) ||
      (values && c->v_cache == nullptr))
    return FA_ERR_INVALID_ARG;
  if ((keys && !aligned_to(c->k_cache, 16)) || (values && !aligned_to(c->v_cache, 16)))
    return FA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->num_pages > (1 << 30) || c->max_pages < 0 ||
      (c->max_pages > 0 && c->block_table == nullptr))
    return FA_ERR_INVALID_ARG;
  if (page_shift(c->page_size) < 0) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

inline fa_status status_of(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// Cache pool as a 3-D tensor (d, page_size, pages x heads): boxes of one page x 64 columns with
// the 128-byte swizzle.  The coordinate num_pages * Hkv lies outside and reads as zeros.
inline bool make_pool_map(CUtensorMap* m, const void* base, const fa_paged_kv& c, int Hkv, int d) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t page = static_cast<cuuint64_t>(c.page_size);
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), page,
                        static_cast<cuuint64_t>(c.num_pages) * static_cast<cuuint64_t>(Hkv)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, page * static_cast<cuuint64_t>(d) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(c.page_size), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace fa
