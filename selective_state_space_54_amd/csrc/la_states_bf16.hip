// Linear attention, bf16: segments' own states, forward and in reverse, in one launch.
#include "la_pass_launch.h"
#include "linear_attention.h"

namespace mssm {
namespace la {
hipError_t pass_states_bf16(const PassArgs& fwd, const PassArgs& rev, hipStream_t stream) {
  return launch_states<uint16_t>(fwd, rev, stream);
}
}  // namespace la
}  // namespace mssm
