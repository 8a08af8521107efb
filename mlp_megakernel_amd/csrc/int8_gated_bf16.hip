// The gated 8-bit product with results of type __bf16.
#include "int8_forward.hpp"

namespace coalesce {

hipError_t launch_int8_gated_bf16(const Int8Params& p, hipStream_t stream, int num_cus, void* workspace) {
  return int8_forward<__bf16, EPI_INT8_GATED>(p, stream, num_cus, workspace);
}

}  // namespace coalesce
