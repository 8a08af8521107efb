// Gated product, f16 inputs (ffn_forward.hpp).
#include "ffn_forward.hpp"

namespace coalesce {

hipError_t launch_gated_f16(const FfnParams& p, DType out, int act, hipStream_t stream, int num_cus, void* workspace) {
  return forward_typed<_Float16, EPI_GATED>(p, DT_F16, out, act, stream, num_cus, workspace);
}

}  // namespace coalesce
