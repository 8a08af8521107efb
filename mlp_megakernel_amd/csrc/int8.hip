// Choice of kernel for the 8-bit products, the partial sums of a split contraction
// and the pass that joins them.
#include "ffn_plan.hpp"
#include "gemm16_core.hpp"

namespace coalesce {
namespace {

// Four consecutive columns of one row per thread and iteration.
template <typename TO>
__global__ __launch_bounds__(256) void int8_join_kernel(Int8Join j) {
  const int64_t quads = (j.q.N + 3) >> 2, total = (int64_t)j.q.M * quads;
  for (int64_t w = (int64_t)blockIdx.x * 256 + threadIdx.x; w < total; w += (int64_t)gridDim.x * 256) {
    const int64_t m = w / quads;
    const int n = (int)(w - m * quads) * 4;
    const int valid = min(4, j.q.N - n);
    const float sa = j.q.scale_a[m];
    f32x4 z[2];
    for (int i = 0; i < j.products; ++i) {
      const int32_t* p = j.P[i] + m * j.ldp + n;
      i32x4 s = (i32x4){0, 0, 0, 0};
      for (int k = 0; k < j.splits; k += 8) {
        i32x4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          v[u] = k + u < j.splits ? *(const i32x4*)(p + (int64_t)(k + u) * j.split_stride) : (i32x4){0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < 8; ++u) s += v[u];
      }
      const f32x4 sb = load4<float>(j.q.scale_b[i] + n, valid);
      const f32x4 b = j.q.bias[i] ? load4<float>((const float*)j.q.bias[i] + n, valid) : (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < 4; ++r) z[i][r] = __builtin_fmaf((float)s[r] * sa, sb[r], b[r]);
    }
    f32x4 o = act_any(j.q.act, z[0]);
    if (j.products == 2)
      o = o * z[1];
    else if (j.q.R)
      o = load4<TO>((const TO*)j.q.R + m * j.q.ldr + n, valid) + o;
    store4<TO>((TO*)j.q.Y + m * j.q.ldy + n, o, valid);
  }
}

template <typename TO>
hipError_t join_t(const Int8Join& j, hipStream_t stream, int num_cus) {
  const int64_t blocks = ((int64_t)j.q.M * ((j.q.N + 3) / 4) + 255) / 256;
  hipLaunchKernelGGL((int8_join_kernel<TO>), dim3((unsigned)std::min<int64_t>(blocks, (int64_t)num_cus * 8)), dim3(256),
                     0, stream, j);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_sums(const TileOp& o, bool gated, int variant, hipStream_t stream, int num_cus) {
  // the int32 sums pass through the fp32 store as they are: moved, never computed with
#define COALESCE_TILE(...) \
  launch_tile<i8pair, float, LAY_K, LAY_K, 1, EPI_STORE, TileGeo<__VA_ARGS__>>(o, stream, num_cus)
  if (gated) return variant == kShape128 ? COALESCE_TILE(128, 128, 4, 2, 2, 2) : COALESCE_TILE(64, 128, 4, 2, 2, 2);
  return variant == kShape128       ? COALESCE_TILE(128, 128, 4, 2, 2, 1)
         : variant == kShape128Deep ? COALESCE_TILE(128, 128, 4, 2, 1, 1, 3)
                                    : COALESCE_TILE(64, 64, 4, 2, 4, 1);
#undef COALESCE_TILE
}

hipError_t launch_int8_join(const Int8Join& j, DType out, hipStream_t stream, int num_cus) {
  if (out == DT_F32) return join_t<float>(j, stream, num_cus);
  return out == DT_BF16 ? join_t<__bf16>(j, stream, num_cus) : join_t<_Float16>(j, stream, num_cus);
}

size_t int8_workspace(int64_t M, int64_t N, int64_t K, bool gated, int num_cus) {
  const Int8Plan f = plan_int8(M, N, K, gated, num_cus);
  return f.few ? 0 : partial_bytes(f.tiles, M, N, gated ? 2 : 1);
}

hipError_t launch_int8(const Int8Params& p, bool gated, DType out, hipStream_t stream, int num_cus, void* workspace) {
  if (out == DT_F32)
    return gated ? launch_int8_gated_f32(p, stream, num_cus, workspace)
                 : launch_int8_resid_f32(p, stream, num_cus, workspace);
  if (out == DT_BF16)
    return gated ? launch_int8_gated_bf16(p, stream, num_cus, workspace)
                 : launch_int8_resid_bf16(p, stream, num_cus, workspace);
  return gated ? launch_int8_gated_f16(p, stream, num_cus, workspace)
               : launch_int8_resid_f16(p, stream, num_cus, workspace);
}

}  // namespace coalesce
