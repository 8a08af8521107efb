// The 8-bit product with residual with results of type _Float16.
#include "int8_forward.hpp"

namespace coalesce {

hipError_t launch_int8_resid_f16(const Int8Params& p, hipStream_t stream, int num_cus, void* workspace) {
  return int8_forward<_Float16, EPI_INT8_RESID>(p, stream, num_cus, workspace);
}

}  // namespace coalesce
