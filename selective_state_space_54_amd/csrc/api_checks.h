// Argument checks that the C-ABI front ends share.  All run before the first HIP call.
#pragma once

#include <initializer_list>
#include <limits>

#include "mssm_internal.h"

namespace mssm {

constexpr int64_t kMaxBlocks = (int64_t(1) << 32) / 256 - 1;   // blocks of 256 threads

inline bool product(std::initializer_list<int64_t> f, int64_t* out) {
  int64_t n = 1;
  for (int64_t v : f) {
    if (v == 0) { *out = 0; return true; }
  }
  for (int64_t v : f) {
    if (n > std::numeric_limits<int64_t>::max() / v) return false;
    n *= v;
  }
  *out = n;
  return true;
}

inline bool bad_dtype(mssm_dtype t) { return t != MSSM_FLOAT32 && t != MSSM_BFLOAT16; }

inline mssm_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return MSSM_SUCCESS;
  if (!ws || have < need || reinterpret_cast<uintptr_t>(ws) % 256 != 0) return MSSM_ERROR_WORKSPACE;
  return MSSM_SUCCESS;
}

// Whether two of the outputs, or an output and an input, begin at one address.
inline bool same_address(std::initializer_list<const void*> outputs,
                         std::initializer_list<const void*> inputs = {}) {
  for (auto a = outputs.begin(); a != outputs.end(); ++a) {
    if (!*a) continue;
    for (auto b = a + 1; b != outputs.end(); ++b)
      if (*a == *b) return true;
    for (const void* b : inputs)
      if (*a == b) return true;
  }
  return false;
}

inline mssm_status done(hipError_t e, const char* where) {
  if (e == hipSuccess) return MSSM_SUCCESS;
  set_hip_error(e, where);
  return MSSM_ERROR_HIP;
}

}  // namespace mssm
