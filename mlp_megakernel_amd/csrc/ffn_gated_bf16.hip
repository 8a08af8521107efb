// Gated product, bf16 inputs (ffn_forward.hpp).
#include "ffn_forward.hpp"

namespace coalesce {

hipError_t launch_gated_bf16(const FfnParams& p, DType out, int act, hipStream_t stream, int num_cus, void* workspace) {
  return forward_typed<__bf16, EPI_GATED>(p, DT_BF16, out, act, stream, num_cus, workspace);
}

}  // namespace coalesce
