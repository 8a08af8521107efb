// The products on 8-bit operands, for one output type:
//   plain  Y = act(z) + R;   gated  Y = act(zg) zu
//   z[m][n] = scale_a[m] scale_b[n] sum_k A[m][k] B[n][k] + bias[n]
// on the tiles of gemm16_core.hpp: the operands travel as pairs of bytes, both
// along the contraction, so a K step of 128 has the bytes, the LDS traffic and the
// matrix-core time of a 16-bit step of 64, for twice the products.  The sums are exact
// in int32 (K up to 131071), so every tile shape, split and the few-row kernel give the
// same bits.
#pragma once
#include "ffn_plan.hpp"
#include "int8_few.hpp"

namespace coalesce {
namespace {

template <typename TO, int EPI>
hipError_t int8_tiles(const TileOp& o, int variant, hipStream_t stream, int num_cus) {
#define COALESCE_TILE(...) launch_tile<i8pair, TO, LAY_K, LAY_K, 1, EPI, TileGeo<__VA_ARGS__>>(o, stream, num_cus)
  if constexpr (EPI == EPI_INT8_GATED) {
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

template <typename TO, int EPI>
hipError_t int8_forward(const Int8Params& q, hipStream_t stream, int num_cus, void* workspace) {
  constexpr bool gated = EPI == EPI_INT8_GATED;
  TileOp o{};
  o.a[0] = q.A;
  o.lda = q.lda / 2;  // in pairs
  o.ldb = q.ldb / 2;
  for (int i = 0; i < 2; ++i) {
    o.b[i] = q.B[i];
    o.bias[i] = q.bias[i];
    o.scale_n[i] = q.scale_b[i];
  }
  o.scale_m = q.scale_a;
  o.M = q.M;
  o.N = q.N;
  o.K = q.K;
  o.batch = o.splits = 1;
  o.R = q.R;
  o.ldr = q.ldr;
  o.Y[0] = q.Y;
  o.ldy = q.ldy;
  o.act = q.act;
  const Int8Plan f = plan_int8(q.M, q.N, q.K, gated, num_cus);
  if (f.few) return launch_few8<TO, EPI>(o, f.few, stream);
  o.splits = f.tiles.splits;
  if (o.splits == 1) return int8_tiles<TO, EPI>(o, f.tiles.variant, stream, num_cus);
  Int8Join j{};
  j.products = gated ? 2 : 1;
  j.ldp = partial_pitch(o.N);
  j.split_stride = (int64_t)o.M * j.ldp;
  j.splits = o.splits;
  const size_t one = align256((size_t)o.splits * (size_t)j.split_stride * 4) / 4;
  for (int i = 0; i < j.products; ++i) {
    j.P[i] = (const int32_t*)workspace + i * one;
    o.Y[i] = (void*)j.P[i];
  }
  o.ldy = j.ldp;
  o.split_stride = j.split_stride;
  hipError_t e = launch_int8_sums(o, gated, f.tiles.variant, stream, num_cus);
  if (e != hipSuccess) return e;
  j.q = q;
  return launch_int8_join(j, sizeof(TO) == 4 ? DT_F32 : __is_same(TO, __bf16) ? DT_BF16 : DT_F16, stream, num_cus);
}

}  // namespace
}  // namespace coalesce
