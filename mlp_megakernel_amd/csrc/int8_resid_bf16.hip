// The 8-bit product with residual with results of type __bf16.
#include "int8_forward.hpp"

namespace coalesce {

hipError_t launch_int8_resid_bf16(const Int8Params& p, hipStream_t stream, int num_cus, void* workspace) {
  return int8_forward<__bf16, EPI_INT8_RESID>(p, stream, num_cus, workspace);
}

}  // namespace coalesce
