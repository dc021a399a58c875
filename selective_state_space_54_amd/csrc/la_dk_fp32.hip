// Linear attention, fp32: dk and dg.
#include "la_pass_launch.h"
#include "linear_attention.h"

namespace mssm {
namespace la {
hipError_t pass_dk_fp32(const PassArgs& p, hipStream_t stream) {
  return launch_pass<float, true, true, 2>(p, stream);
}
}  // namespace la
}  // namespace mssm
