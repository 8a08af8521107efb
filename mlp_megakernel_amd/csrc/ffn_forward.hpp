// Forward of the feed-forward operators on gfx950 MFMA, for one input type:
//   gated product       H = act(X Wg + bg) * (X Wu + bu)
//   GEMM with residual  Y = act(X W + bias) + R
// Both products of the gated form share every fragment of X: a workgroup tile
// holds the same columns of both, so the activation, the product and one
// rounding happen on the accumulators and neither projection is written
// (unless a training forward asks for the pre-activations).  Compiled per
// input type and operator (ffn_gated_*.hip, ffn_resid_*.hip).
#pragma once
#include "ffn_few.hpp"
#include "ffn_plan.hpp"
#include "gemm16_core.hpp"

namespace coalesce {
namespace {

template <typename T, typename TO, int EPI>
hipError_t forward_tiles(const TileOp& o, int variant, hipStream_t stream, int num_cus) {
#define COALESCE_TILE(...) launch_tile<T, TO, LAY_K, LAY_X, 1, EPI, TileGeo<__VA_ARGS__>>(o, stream, num_cus)
  if constexpr (EPI == EPI_GATED) {
    // 256 rows x 128 columns of both products: waves of 64 x (64 + 64); 224,
    // 192 and 160 rows: waves of half of them x (32 + 32); 128 x 64: waves of
    // 64 x (32 + 32); 64 x 64: waves of 32 x (32 + 32)
    switch (variant) {
      case kShape256: return COALESCE_TILE(256, 256, 8, 4, 1, 2);
      case kShape224: return COALESCE_TILE(224, 256, 8, 2, 1, 2);
      case kShape192: return COALESCE_TILE(192, 256, 8, 2, 1, 2);
      case kShape160: return COALESCE_TILE(160, 256, 8, 2, 1, 2, 3);
      case kShape128: return COALESCE_TILE(128, 128, 4, 2, 2, 2);
      default: return COALESCE_TILE(64, 128, 4, 2, 2, 2);
    }
  } else {
    switch (variant) {
      case kShape256: return COALESCE_TILE(256, 256, 8, 2, 1, 1);
      case kShape224: return COALESCE_TILE(224, 256, 8, 2, 1, 1);
      case kShape192: return COALESCE_TILE(192, 256, 8, 2, 1, 1);
      case kShape160: return COALESCE_TILE(160, 256, 8, 2, 1, 1, 3);
      case kShape128: return COALESCE_TILE(128, 128, 4, 2, 2, 1);
      case kShape128Deep: return COALESCE_TILE(128, 128, 4, 2, 1, 1, 3);
      case kShape64Deep: return COALESCE_TILE(64, 64, 4, 2, 3, 1, 3);
      default: return COALESCE_TILE(64, 64, 4, 2, 4, 1);
    }
  }
#undef COALESCE_TILE
}

// A split product: fp32 partial results of each range of K steps (128 x 128 or
// 64 x 64 tiles), summed and finished by the combining pass.
template <typename T, int EPI>
hipError_t forward_split(TileOp o, int variant, DType in, DType out, int act, hipStream_t stream, int num_cus,
                         float* ws) {
  CombineOp c{};
  const int products = EPI == EPI_GATED ? 2 : 1;
  c.ldp = partial_pitch(o.N);
  c.split_stride = (int64_t)o.M * c.ldp;
  c.splits = o.splits;
  c.products = products;
  const size_t one = align256((size_t)o.splits * (size_t)c.split_stride * 4) / 4;
  for (int i = 0; i < products; ++i) {
    c.P[i] = ws + i * one;
    c.bias[i] = o.bias[i];
    c.Z[i] = o.Z[i];
  }
  c.R = o.R;
  c.ldr = o.ldr;
  c.ldz = o.ldz;
  c.Y[0] = o.Y[0];
  c.ldy = o.ldy;
  c.M = o.M;
  c.N = o.N;
  c.act = act;
  for (int i = 0; i < products; ++i) o.Y[i] = (void*)c.P[i];
  o.ldy = c.ldp;
  o.split_stride = c.split_stride;
#define COALESCE_TILE(...) launch_tile<T, float, LAY_K, LAY_X, 1, EPI_STORE, TileGeo<__VA_ARGS__>>(o, stream, num_cus)
  hipError_t e;
  if constexpr (EPI == EPI_GATED)
    e = variant == kShape128 ? COALESCE_TILE(128, 128, 4, 2, 2, 2) : COALESCE_TILE(64, 128, 4, 2, 2, 2);
  else
    e = variant == kShape128       ? COALESCE_TILE(128, 128, 4, 2, 2, 1)
        : variant == kShape128Deep ? COALESCE_TILE(128, 128, 4, 2, 1, 1, 3)
                                   : COALESCE_TILE(64, 64, 4, 2, 4, 1);
#undef COALESCE_TILE
  if (e != hipSuccess) return e;
  return launch_combine(c, EPI == EPI_GATED ? COMBINE_GATED : COMBINE_RESID, in, out, stream, num_cus);
}

template <typename T, int EPI>
hipError_t forward_typed(const FfnParams& p, DType in, DType out, int act, hipStream_t stream, int num_cus,
                         void* workspace) {
  TileOp o{};
  o.a[0] = p.X;
  o.lda = p.ldx;
  o.ldb = p.ldw;
  for (int i = 0; i < 2; ++i) {
    o.b[i] = p.W[i];
    o.bias[i] = p.bias[i];
    o.Z[i] = p.Z[i];
  }
  o.M = p.M;
  o.N = p.N;
  o.K = p.K;
  o.batch = o.splits = 1;
  o.R = p.R;
  o.ldr = p.ldr;
  o.ldz = p.ldz;
  o.Y[0] = p.Y;
  o.ldy = p.ldy;
  o.act = act;
  const ForwardPlan f = plan_forward(p.M, p.N, p.K, EPI == EPI_GATED, num_cus);
  if (f.strip)
    return out == DT_F32 ? launch_few<T, float, EPI>(o, f.strip, stream) : launch_few<T, T, EPI>(o, f.strip, stream);
  const TilePlan& plan = f.tiles;
  o.splits = plan.splits;
  if (plan.splits > 1)
    return forward_split<T, EPI>(o, plan.variant, in, out, act, stream, num_cus, (float*)workspace);
  if (out == DT_F32) return forward_tiles<T, float, EPI>(o, plan.variant, stream, num_cus);
  return forward_tiles<T, T, EPI>(o, plan.variant, stream, num_cus);
}

}  // namespace
}  // namespace coalesce
