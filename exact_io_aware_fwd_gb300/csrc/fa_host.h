// Host helpers that every C-ABI translation unit uses (defined in fa_api.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cudaTypedefs.h>

#include "fa.h"

namespace fa {

int* status_ptr();           // this device's status word, or nullptr
uint64_t wait_timeout_ns();  // limit of a single pipeline wait
fa_status check_device();    // the current device is an sm_103 part
fa_status check_workspace(void* ws, size_t bytes, size_t need);
float resolve_scale(float scale, int d);         // scale < 0: 1/sqrt(d)
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();   // cuTensorMapEncodeTiled, or nullptr

inline bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

}  // namespace fa
