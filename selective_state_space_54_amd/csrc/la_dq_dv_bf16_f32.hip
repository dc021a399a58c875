// Linear attention, bf16: dq, kept in float32 to be summed over heads, and dv.
#include "la_pass_launch.h"
#include "linear_attention.h"

namespace mssm {
namespace la {
hipError_t pass_dq_dv_bf16_f32(const PassArgs& dq, const PassArgs& dv, hipStream_t stream) {
  return launch_dq_dv<uint16_t, float>(dq, dv, stream);
}
}  // namespace la
}  // namespace mssm
