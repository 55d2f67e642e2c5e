// Argument checks that the rollout side's entry points share.
#pragma once

#include <cstdint>

#include "../../include/sinkattn.h"
#include "internal.h"

namespace sa {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline sinkattn_status from_cuda(cudaError_t e) { return e == cudaSuccess ? SINKATTN_OK : SINKATTN_ERR_CUDA; }

// A list of n slots (or other int32 per request).
inline sinkattn_status check_list(int32_t n, const void* list) {
  if (n < 0) return SINKATTN_ERR_INVALID_ARG;
  if (n > kKv4MaxRequests) return SINKATTN_ERR_UNSUPPORTED;
  if (n > 0 && !list) return SINKATTN_ERR_INVALID_ARG;
  if (!aligned4(list)) return SINKATTN_ERR_ALIGNMENT;
  return SINKATTN_OK;
}

}  // namespace sa
