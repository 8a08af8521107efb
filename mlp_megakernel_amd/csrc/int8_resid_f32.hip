// The 8-bit product with residual with results of type float.
#include "int8_forward.hpp"

namespace coalesce {

hipError_t launch_int8_resid_f32(const Int8Params& p, hipStream_t stream, int num_cus, void* workspace) {
  return int8_forward<float, EPI_INT8_RESID>(p, stream, num_cus, workspace);
}

}  // namespace coalesce
