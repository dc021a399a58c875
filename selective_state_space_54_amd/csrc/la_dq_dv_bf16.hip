// Linear attention, bf16: dq with the queries' part of dg, and dv.
#include "la_pass_launch.h"
#include "linear_attention.h"

namespace mssm {
namespace la {
hipError_t pass_dq_dv_bf16(const PassArgs& dq, const PassArgs& dv, hipStream_t stream) {
  return launch_dq_dv<uint16_t, uint16_t>(dq, dv, stream);
}
}  // namespace la
}  // namespace mssm
