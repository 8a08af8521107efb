// Backward of the feed-forward operators, bf16 inputs (ffn_backward.hpp).
#include "ffn_backward.hpp"

namespace coalesce {

hipError_t launch_backward_bf16(const FfnBwdParams& p, bool gated, DType dy, DType grad, int act, hipStream_t stream,
                              int num_cus, void* workspace) {
  return backward_typed<__bf16>(p, DT_BF16, gated, dy, grad, act, stream, num_cus, workspace);
}

}  // namespace coalesce
