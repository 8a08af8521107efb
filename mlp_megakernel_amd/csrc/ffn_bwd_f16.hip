// Backward of the feed-forward operators, f16 inputs (ffn_backward.hpp).
#include "ffn_backward.hpp"

namespace coalesce {

hipError_t launch_backward_f16(const FfnBwdParams& p, bool gated, DType dy, DType grad, int act, hipStream_t stream,
                              int num_cus, void* workspace) {
  return backward_typed<_Float16>(p, DT_F16, gated, dy, grad, act, stream, num_cus, workspace);
}

}  // namespace coalesce
