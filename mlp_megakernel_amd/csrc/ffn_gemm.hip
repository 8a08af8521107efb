// Forward of the feed-forward operators on gfx950 MFMA:
//   gated product       H = act(X Wg + bg) * (X Wu + bu)
//   GEMM with residual  Y = act(X W + bias) + R
// Both products of the gated form share every fragment of X: a workgroup tile
// holds the same columns of both, so the activation, the product and one
// rounding happen on the accumulators and neither projection is written
// (unless a training forward asks for the pre-activations).
#include "gemm16_core.hpp"

namespace coalesce {
namespace {

typedef TileGeo<128, 128, 4, 2, 2, 1> Geo128;
typedef TileGeo<128, 128, 4, 2, 2, 2> GeoG128;

TileOp forward_op(const FfnParams& p, int act) {
  TileOp o{};
  o.a[0] = p.X;
  o.lda[0] = p.ldx;
  for (int i = 0; i < 2; ++i) {
    o.b[i] = p.W[i];
    o.ldb[i] = p.ldw[i];
    o.bias[i] = p.bias[i];
    o.Z[i] = p.Z[i];
  }
  o.M = p.M;
  o.N = p.N;
  o.K = p.K;
  o.segs = o.batch = o.splits = 1;
  o.R = p.R;
  o.ldr = p.ldr;
  o.ldz = p.ldz;
  o.Y[0] = p.Y;
  o.ldy[0] = p.ldy;
  o.act = act;
  return o;
}

template <typename T, typename TO>
hipError_t forward_t(const FfnParams& p, bool gated, int act, hipStream_t stream, int num_cus) {
  const TileOp o = forward_op(p, act);
  if (gated) return launch_tile<T, TO, LAY_K, LAY_X, EPI_GATED, GeoG128>(o, stream, num_cus);
  return launch_tile<T, TO, LAY_K, LAY_X, EPI_RESID, Geo128>(o, stream, num_cus);
}

}  // namespace

size_t ffn_forward_workspace(int64_t, int64_t, int64_t, bool, int) { return 0; }

hipError_t launch_ffn_forward(const FfnParams& p, bool gated, DType in, DType out, int act, hipStream_t stream,
                              int num_cus, void*) {
  if (in == DT_BF16) {
    if (out == DT_F32) return forward_t<__bf16, float>(p, gated, act, stream, num_cus);
    return forward_t<__bf16, __bf16>(p, gated, act, stream, num_cus);
  }
  if (out == DT_F32) return forward_t<_Float16, float>(p, gated, act, stream, num_cus);
  return forward_t<_Float16, _Float16>(p, gated, act, stream, num_cus);
}

}  // namespace coalesce
