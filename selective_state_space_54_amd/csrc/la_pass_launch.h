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

template <typename T, int DA, int NT, int kHeads>
hipError_t launch_states_as(const PassArgs& fwd, const PassArgs& rev, hipStream_t stream) {
  const int64_t blocks = fwd.grid.slots * (fwd.heads / kHeads);
  hipLaunchKernelGGL((la_states<T, sizeof(T) == 2 ? 64 : 32, DA, NT, kHeads>),
                     dim3(static_cast<uint32_t>(blocks), 2), dim3(kThreads), 0, stream, fwd, rev);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_states(const PassArgs& fwd, const PassArgs& rev, hipStream_t stream) {
  if (fwd.paired)
    return fwd.dA <= 64 ? launch_states_as<T, 64, 2, 2>(fwd, rev, stream)
                        : launch_states_as<T, 128, 2, 2>(fwd, rev, stream);
  if (fwd.dA <= 64)
    return fwd.dB <= 64 ? launch_states_as<T, 64, 1, 1>(fwd, rev, stream)
                        : launch_states_as<T, 64, 2, 1>(fwd, rev, stream);
  return fwd.dB <= 64 ? launch_states_as<T, 128, 1, 1>(fwd, rev, stream)
                      : launch_states_as<T, 128, 2, 1>(fwd, rev, stream);
}

template <typename T, typename V, int DK, int DV, int kHeads>
hipError_t launch_dq_dv_as(const PassArgs& dq, const PassArgs& dv, hipStream_t stream) {
  const int64_t n = dq.grid.slots * dq.heads;
  hipLaunchKernelGGL((la_dq_dv<T, V, sizeof(T) == 2 ? 64 : 32, DK, DV, kHeads>),
                     dim3(static_cast<uint32_t>(n + n / kHeads)), dim3(kThreads), 0, stream, dq, dv,
                     static_cast<uint32_t>(n));
  return hipGetLastError();
}

template <typename T, typename V>
hipError_t launch_dq_dv(const PassArgs& dq, const PassArgs& dv, hipStream_t stream) {
  if (dv.paired)
    return dv.dA <= 64 ? launch_dq_dv_as<T, V, 64, 64, 2>(dq, dv, stream)
                       : launch_dq_dv_as<T, V, 128, 64, 2>(dq, dv, stream);
  if (dv.dA <= 64)
    return dv.dB <= 64 ? launch_dq_dv_as<T, V, 64, 64, 1>(dq, dv, stream)
                       : launch_dq_dv_as<T, V, 64, 128, 1>(dq, dv, stream);
  return dv.dB <= 64 ? launch_dq_dv_as<T, V, 128, 64, 1>(dq, dv, stream)
                     : launch_dq_dv_as<T, V, 128, 128, 1>(dq, dv, stream);
}

}  // namespace la
}  // namespace mssm
