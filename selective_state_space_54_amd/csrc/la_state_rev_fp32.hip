// Linear attention, fp32: a segment's own adjoint state.
#include "la_pass_launch.h"
#include "linear_attention.h"

namespace mssm {
namespace la {
hipError_t pass_state_rev_fp32(const PassArgs& p, hipStream_t stream) {
  return launch_pass<float, true, false, 0>(p, stream);
}
}  // namespace la
}  // namespace mssm
