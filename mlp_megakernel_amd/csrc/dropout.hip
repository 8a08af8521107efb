// Dropout on gfx950: Y = R + keep(X) / (1 - p), or without R; its gradient is
// the same operation on dY.  The mask comes from the generator (philox.hpp) and is
// never stored.  Bound by memory with a residual; without one the generator's 20
// products of 64 bits per 8 values take about as long.  8 columns per thread, one
// access each: many short-lived workgroups keep more loads in flight than few
// long-lived ones (8192 x 16384 bf16: 90 us so, 97 and 100 with grids of 8192 and
// 2048 workgroups that walk on).
#include "philox.hpp"
#include "rows.hpp"

namespace coalesce {
namespace {

// A workgroup covers 2^lg 8-column pieces of 256 >> lg rows.
template <typename T, typename TO>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutParams p, int lg, int col_blocks) {
  const uint32_t block = (uint32_t)block_no(), band_no = block / (uint32_t)col_blocks;  // (2^41 elements: 2^31 blocks)
  const int64_t band = band_no;
  const int part = (int)(block - band_no * (uint32_t)col_blocks);
  const int64_t row = band * (256 >> lg) + (threadIdx.x >> lg);
  const int n = ((part << lg) + (int)(threadIdx.x & ((1 << lg) - 1))) * 8;
  if (row >= p.M || n >= p.N) return;
  const DropKey key = drop_key(p.drop);
  const int valid = p.N - n;
  float v[8], r[8];
  auto read = [&](auto* src, float (&x)[8]) {
    typedef __typeof__(*src) E;
    typedef E e4 __attribute__((ext_vector_type(16 / sizeof(E))));
    constexpr int W = 16 / sizeof(E);
    // whole 16-byte pieces that hold at least one column of the row
#pragma unroll
    for (int i = 0; i < 8 / W; ++i) {
      e4 t{};
      if (i * W < valid) t = *(const e4*)(src + i * W);
#pragma unroll
      for (int e = 0; e < W; ++e) x[i * W + e] = (float)t[e];
    }
  };
  read((T*)p.X + row * p.ldx + n, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = 0.0f;
  if (p.R) read((TO*)p.R + row * p.ldr + n, r);
  if (p.drop.on) drop8(key, (uint32_t)row, (uint32_t)n, v);
  // without a residual nothing is added (0 + -0 would lose the sign)
  if (p.R) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += r[e];
  }
  TO* dst = (TO*)p.Y + row * p.ldy + n;
  if (valid >= 8) {
    constexpr int W = 16 / sizeof(TO);
    typedef TO e4 __attribute__((ext_vector_type(16 / sizeof(TO))));
#pragma unroll
    for (int i = 0; i < 8 / W; ++i) {
      e4 t;
#pragma unroll
      for (int e = 0; e < W; ++e) t[e] = (TO)v[i * W + e];
      *(e4*)(dst + i * W) = t;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < valid) dst[e] = (TO)v[e];
  }
}

template <typename T, typename TO>
hipError_t dropout_typed(const DropoutParams& p, hipStream_t stream) {
  const int64_t pieces = ((int64_t)p.N + 7) / 8;
  int lg = 0;
  while (lg < 8 && ((int64_t)1 << lg) < pieces) ++lg;
  const int64_t col_blocks = (pieces + ((int64_t)1 << lg) - 1) >> lg, rows = 256 >> lg;
  const int64_t bands = (p.M + rows - 1) / rows;
  hipLaunchKernelGGL((dropout_kernel<T, TO>), blocks_grid(bands * col_blocks), dim3(256), 0, stream, p, lg,
                     (int)col_blocks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutParams& p, DType in, DType out, hipStream_t stream) {
  if (in == DT_F32) return dropout_typed<float, float>(p, stream);
  if (in == DT_BF16)
    return out == DT_F32 ? dropout_typed<__bf16, float>(p, stream) : dropout_typed<__bf16, __bf16>(p, stream);
  return out == DT_F32 ? dropout_typed<_Float16, float>(p, stream) : dropout_typed<_Float16, _Float16>(p, stream);
}

}  // namespace coalesce
