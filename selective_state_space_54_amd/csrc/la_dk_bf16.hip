// Linear attention, bf16: dk and dg.
#include "la_pass_launch.h"
#include "linear_attention.h"

namespace mssm {
namespace la {
hipError_t pass_dk_bf16(const PassArgs& p, hipStream_t stream) {
  return launch_pass<uint16_t, true, true, 2>(p, stream);
}
}  // namespace la
}  // namespace mssm
