// Linear attention, bf16: dq, and the queries' part of dg.
#include "la_pass_launch.h"
#include "linear_attention.h"

namespace mssm {
namespace la {
hipError_t pass_dq_bf16(const PassArgs& p, hipStream_t stream) {
  return launch_pass<uint16_t, false, true, 1>(p, stream);
}
}  // namespace la
}  // namespace mssm
