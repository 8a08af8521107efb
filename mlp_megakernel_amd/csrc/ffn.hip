// Choice of kernel for the feed-forward operators, and the pass that combines
// the ranges of a split product.
#include "ffn_plan.hpp"
#include "gemm16_core.hpp"

namespace coalesce {
namespace {

// Four consecutive columns of one row per thread and iteration; the ranges are
// added in order, so the result does not depend on timing.
template <typename T, typename TO, int KIND>
__global__ __launch_bounds__(256) void combine_kernel(CombineOp c) {
  const int64_t quads = (c.N + 3) >> 2, total = (int64_t)c.M * quads;
  const int i0 = KIND == COMBINE_STORE ? blockIdx.y : 0;
  for (int64_t w = (int64_t)blockIdx.x * 256 + threadIdx.x; w < total; w += (int64_t)gridDim.x * 256) {
    const int64_t m = w / quads;
    const int n = (int)(w - m * quads) * 4;
    const int valid = min(4, c.N - n);
    f32x4 acc[2];
#pragma unroll
    for (int i = 0; i < (KIND == COMBINE_GATED ? 2 : 1); ++i) {
      const float* p = c.P[i + i0] + m * c.ldp + n;
      // eight loads in flight: the results come from other XCDs' writes
      f32x4 s = (f32x4){0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < c.splits; k += 8) {
        f32x4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          v[u] = k + u < c.splits ? *(const f32x4*)(p + (int64_t)(k + u) * c.split_stride)
                                  : (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < 8; ++u) s += v[u];
      }
      acc[i] = s;
    }
    if constexpr (KIND == COMBINE_STORE) {
      store4<TO>((TO*)c.Y[i0] + m * c.ldy + n, acc[0], valid);
    } else {
#pragma unroll
      for (int i = 0; i < (KIND == COMBINE_GATED ? 2 : 1); ++i) {
        if (c.bias[i]) acc[i] += load4<T>((const T*)c.bias[i] + n, valid);
        if (c.Z[i]) store4<T>((T*)c.Z[i] + m * c.ldz + n, acc[i], valid);
      }
      f32x4 o = (f32x4){0.f, 0.f, 0.f, 0.f};
      if (KIND == COMBINE_RESID && c.R) o = load4<TO>((const TO*)c.R + m * c.ldr + n, valid);
      const f32x4 f = act_any(c.act, acc[0]);
      o = KIND == COMBINE_GATED ? f * acc[1] : o + f;
      store4<TO>((TO*)c.Y[0] + m * c.ldy + n, o, valid);
    }
  }
}

template <typename T, typename TO, int KIND>
hipError_t combine_t(const CombineOp& c, hipStream_t stream, int num_cus) {
  const int64_t blocks = ((int64_t)c.M * ((c.N + 3) / 4) + 255) / 256;
  const dim3 grid((unsigned)std::min<int64_t>(blocks, (int64_t)num_cus * 8),
                  KIND == COMBINE_STORE ? (unsigned)c.products : 1u);
  hipLaunchKernelGGL((combine_kernel<T, TO, KIND>), grid, dim3(256), 0, stream, c);
  return hipGetLastError();
}

// An epilogue of one input type, to that type or fp32.
template <typename T, int KIND>
hipError_t combine_in(const CombineOp& c, DType out, hipStream_t stream, int num_cus) {
  return out == DT_F32 ? combine_t<T, float, KIND>(c, stream, num_cus) : combine_t<T, T, KIND>(c, stream, num_cus);
}

}  // namespace

hipError_t launch_combine(const CombineOp& c, CombineKind kind, DType in, DType out, hipStream_t stream, int num_cus) {
  if (kind == COMBINE_STORE) {  // no bias, activation or residual: the inputs' type does not matter
    if (out == DT_F32) return combine_t<float, float, COMBINE_STORE>(c, stream, num_cus);
    return out == DT_BF16 ? combine_t<__bf16, __bf16, COMBINE_STORE>(c, stream, num_cus)
                          : combine_t<_Float16, _Float16, COMBINE_STORE>(c, stream, num_cus);
  }
  if (kind == COMBINE_RESID)
    return in == DT_BF16 ? combine_in<__bf16, COMBINE_RESID>(c, out, stream, num_cus)
                         : combine_in<_Float16, COMBINE_RESID>(c, out, stream, num_cus);
  return in == DT_BF16 ? combine_in<__bf16, COMBINE_GATED>(c, out, stream, num_cus)
                       : combine_in<_Float16, COMBINE_GATED>(c, out, stream, num_cus);
}

size_t ffn_forward_workspace(int64_t M, int64_t N, int64_t K, bool gated, int num_cus) {
  return partial_bytes(plan_forward(M, N, K, gated, num_cus).tiles, M, N, gated ? 2 : 1);
}

hipError_t launch_ffn_forward(const FfnParams& p, bool gated, DType in, DType out, int act, hipStream_t stream,
                              int num_cus, void* workspace) {
  if (in == DT_BF16) {
    if (gated) return launch_gated_bf16(p, out, act, stream, num_cus, workspace);
    return launch_resid_bf16(p, out, act, stream, num_cus, workspace);
  }
  if (gated) return launch_gated_f16(p, out, act, stream, num_cus, workspace);
  return launch_resid_f16(p, out, act, stream, num_cus, workspace);
}

size_t ffn_backward_workspace(int64_t M, int64_t N, int64_t K, bool gated, int num_cus) {
  return bwd_plan(M, N, K, gated, num_cus).total;
}

hipError_t launch_ffn_backward(const FfnBwdParams& p, bool gated, DType in, DType dy, DType grad, int act,
                               hipStream_t stream, int num_cus, void* workspace) {
  if (in == DT_BF16) return launch_backward_bf16(p, gated, dy, grad, act, stream, num_cus, workspace);
  return launch_backward_f16(p, gated, dy, grad, act, stream, num_cus, workspace);
}

}  // namespace coalesce
