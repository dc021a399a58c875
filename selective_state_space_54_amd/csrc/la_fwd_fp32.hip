// Linear attention, fp32: the output, forward in time.
#include "la_pass_launch.h"
#include "linear_attention.h"

namespace mssm {
namespace la {
hipError_t pass_fwd_fp32(const PassArgs& p, hipStream_t stream) {
  return launch_pass<float, false, true, 0>(p, stream);
}
}  // namespace la
}  // namespace mssm
