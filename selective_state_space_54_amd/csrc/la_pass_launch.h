// Picks the instance of la_pass for the sizes of a call.
#pragma once

#include "linear_attention.h"
#include "mssm_internal.h"

namespace mssm {
namespace la {

template <typename T, typename V, int DA, int NT, int kHeads, bool kRev, bool kOut, int kDot>
hipError_t launch_pass_as(const PassArgs& p, hipStream_t stream) {
  constexpr int C = sizeof(T) == 2 ? 64 : 32;
  const int64_t blocks = p.grid.slots * (p.heads / kHeads);
  hipLaunchKernelGGL((la_pass<T, V, C, DA, NT, kHeads, kRev, kOut, kDot>),
                     dim3(static_cast<uint32_t>(blocks)), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

template <typename T, typename V, bool kRev, bool kOut, int kDot>
hipError_t launch_pass_to(const PassArgs& p, hipStream_t stream) {
  if constexpr (kDot == 0) {
    if (p.paired)
      return p.dA <= 64 ? launch_pass_as<T, V, 64, 2, 2, kRev, kOut, kDot>(p, stream)
                        : launch_pass_as<T, V, 128, 2, 2, kRev, kOut, kDot>(p, stream);
  }
  if (p.dA <= 64)
    return p.dB <= 64 ? launch_pass_as<T, V, 64, 1, 1, kRev, kOut, kDot>(p, stream)
                      : launch_pass_as<T, V, 64, 2, 1, kRev, kOut, kDot>(p, stream);
  return p.dB <= 64 ? launch_pass_as<T, V, 128, 1, 1, kRev, kOut, kDot>(p, stream)
                    : launch_pass_as<T, V, 128, 2, 1, kRev, kOut, kDot>(p, stream);
}

template <typename T, bool kRev, bool kOut, int kDot>
hipError_t launch_pass(const PassArgs& p, hipStream_t stream) {
  if constexpr (kDot != 0 && sizeof(T) == 2) {
    if (p.out_f32) return launch_pass_to<T, float, kRev, kOut, kDot>(p, stream);
  }
  return launch_pass_to<T, T, kRev, kOut, kDot>(p, stream);
}

}  // namespace la
}  // namespace mssm
