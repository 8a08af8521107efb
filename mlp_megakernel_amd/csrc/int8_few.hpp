// The 8-bit products for few rows (up to 64 tokens): what costs there is reading
// the weights once.
//
// The weights lie channel by channel (N x K), so a fragment of the matrix
// instruction is 16 consecutive bytes of a row in memory: no LDS, no transposing.
// A workgroup owns 16 NT channels (of both matrices of a gated product) and
// deals the K steps of 64 SL bytes to its waves in turn; a wave loads a step's fragments
// straight into registers, one step ahead of the products, and never meets a barrier
// until the end, where the waves' int32 sums meet in LDS.  Integer sums do not depend
// on their order, so a row's result is the one that any other kernel gives.
// Rows past M and channels past N read as zero by the buffers' ranges; k past K
// inside a row of X is masked, which settles it for the weights too.
#pragma once
#include "gemm16_core.hpp"

namespace coalesce {
namespace {

// NB matrices, NT blocks of 16 channels of each, MT blocks of 16 rows, SL slices
// of 64 k per step, NW waves.
template <int NB_, int NT_, int MT_, int SL_, int NW_>
struct Few8Geo {
  static constexpr int NB = NB_, NT = NT_, MT = MT_, SL = SL_, NW = NW_, KB = NB * NT, STEP = 64 * SL;
  static_assert(NW * KB * MT <= 144, "the sums exceed the LDS");
};

template <typename G>
struct Few8Step {
  u32x4 b[G::KB][G::SL], x[G::MT][G::SL];
};

template <typename TO, int EPI, typename G>
__global__ __launch_bounds__(G::NW * 64) void few8_kernel(TileOp p) {
  constexpr int NB = G::NB, NT = G::NT, MT = G::MT, SL = G::SL, NW = G::NW, KB = G::KB;
  __shared__ __attribute__((aligned(16))) i32x4 sums[NW][MT][KB][64];
  const int lane = threadIdx.x & 63, q = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (int)blockIdx.x * 16 * NT;
  const int steps = (p.K + G::STEP - 1) / G::STEP;
  const uint32_t row_bytes = (uint32_t)((p.K + 15) & ~15);
  const uint32_t lda = (uint32_t)p.lda * 2u, ldb = (uint32_t)p.ldb * 2u;  // pitches count pairs

  // 16 rows of a matrix from row r0 on, as far as it has them.
  auto rows16 = [&](const void* base, uint32_t ld, int64_t r0, int all) {
    const int left = (int)min((int64_t)16, (int64_t)all - r0);
    return __builtin_amdgcn_make_buffer_rsrc((void*)((const char*)base + (left > 0 ? r0 : 0) * (int64_t)ld), 0,
                                             left > 0 ? (uint32_t)(left - 1) * ld + row_bytes : 0u, 0x00020000);
  };
  __amdgpu_buffer_rsrc_t rb[KB], rx[MT];
#pragma unroll
  for (int i = 0; i < KB; ++i) rb[i] = rows16(p.b[i / NT], ldb, n0 + 16 * (i % NT), p.N);
#pragma unroll
  for (int m = 0; m < MT; ++m) rx[m] = rows16(p.a[0], lda, 16 * m, p.M);
  const int ob = (int)((uint32_t)q * ldb) + 16 * g, ox = (int)((uint32_t)q * lda) + 16 * g;

  // (the whole offset per lane: a range is checked against that)
  auto load = [&](int s, Few8Step<G>& f) {
    const int kb = ob + s * G::STEP, kx = ox + s * G::STEP;
#pragma unroll
    for (int i = 0; i < KB; ++i)
#pragma unroll
      for (int j = 0; j < SL; ++j)
        f.b[i][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rb[i], kb + 64 * j, 0, 0));
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < SL; ++j)
        f.x[m][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx[m], kx + 64 * j, 0, 0));
  };

  i32x4 acc[KB][MT];
#pragma unroll
  for (int i = 0; i < KB; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = (i32x4){0, 0, 0, 0};
  Few8Step<G> f, nx;
  if (w < steps) load(w, f);
  for (int s = w; s < steps; s += NW) {
    if (s + NW < steps) load(s + NW, nx);
    if ((s + 1) * G::STEP > p.K) {
#pragma unroll
      for (int j = 0; j < SL; ++j) {
        const int left = p.K - s * G::STEP - 64 * j - 16 * g;  // valid bytes of this lane's sixteen
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int n = left - 4 * d;
          const uint32_t mask = n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
#pragma unroll
          for (int m = 0; m < MT; ++m) f.x[m][j][d] &= mask;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < SL; ++j)
#pragma unroll
      for (int i = 0; i < KB; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[i][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, f.b[i][j]),
                                                            __builtin_bit_cast(i32x4, f.x[m][j]), acc[i][m], 0, 0, 0);
    f = nx;
  }

#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < KB; ++i) sums[w][m][i][lane] = acc[i][m];
  __syncthreads();
  // unit of the rest: one 16 x 16 block of the output
  for (int u = w; u < MT * NT; u += NW) {
    const int m = u / NT, t = u % NT;
    const int row = 16 * m + q, n = n0 + 16 * t + 4 * g;
    if (row >= p.M || n >= p.N) continue;
    const int valid = min(4, p.N - n);
    const float sa = p.scale_m[row];
    f32x4 z[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      i32x4 a = sums[0][m][i * NT + t][lane];
#pragma unroll
      for (int v = 1; v < NW; ++v) a += sums[v][m][i * NT + t][lane];
      const f32x4 sb = load4<float>(p.scale_n[i] + n, valid);
      const f32x4 b = p.bias[i] ? load4<float>((const float*)p.bias[i] + n, valid) : (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < 4; ++r) z[i][r] = __builtin_fmaf((float)a[r] * sa, sb[r], b[r]);
    }
    f32x4 o = act_any(p.act, z[0]);
    if constexpr (EPI == EPI_INT8_GATED)
      o = o * z[NB - 1];
    else if (p.R)
      o = load4<TO>((const TO*)p.R + (int64_t)row * p.ldr + n, valid) + o;
    store4<TO>((TO*)p.Y[0] + (int64_t)row * p.ldy + n, o, valid);
  }
}

template <typename TO, int EPI, typename G>
hipError_t few8_launch(const TileOp& o, hipStream_t stream) {
  hipLaunchKernelGGL((few8_kernel<TO, EPI, G>), dim3((unsigned)((o.N + 16 * G::NT - 1) / (16 * G::NT))),
                     dim3(G::NW * 64), 0, stream, o);
  return hipGetLastError();
}

template <typename TO, int EPI>
hipError_t launch_few8(const TileOp& o, hipStream_t stream) {
  constexpr int NB = EPI == EPI_INT8_GATED ? 2 : 1;
  if (o.M <= 16) return few8_launch<TO, EPI, Few8Geo<NB, 1, 1, 4, 8>>(o, stream);
  if (o.M <= 32) return few8_launch<TO, EPI, Few8Geo<NB, 1, 2, 4, 8>>(o, stream);
  return few8_launch<TO, EPI, Few8Geo<NB, 1, 4, 2, 8>>(o, stream);
}

}  // namespace
}  // namespace coalesce
