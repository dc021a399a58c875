// Linear attention, float32: segments' own states, forward and in reverse, in one launch.
#include "la_pass_launch.h"
#include "linear_attention.h"

namespace mssm {
namespace la {
hipError_t pass_states_fp32(const PassArgs& fwd, const PassArgs& rev, hipStream_t stream) {
  return launch_states<float>(fwd, rev, stream);
}
}  // namespace la
}  // namespace mssm
