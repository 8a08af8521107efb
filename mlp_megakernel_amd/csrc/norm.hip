// Layer norm of a residual stream on gfx950, alone or of the sum that it first
// forms and writes:
//   s = R + keep(X) / (1 - p)   (or s = X)
//   y = (s - mean) rstd w + b,  mean = sum s / N,  rstd = 1 / sqrt(sum (s - mean)^2 / N + eps)
// Memory is what bounds it, so each row is read once: its values stay in
// registers, and all of it is fp32 until the one rounding of each result.  The mean
// comes first, then the squares of the deviations from it (a sum of squares less a
// squared mean would cancel where the mean is large).  The sum's roundings leave the
// mean off by some steps of the values' size, which is nothing beside the deviations
// unless the mean is larger than those (a constant row of 1e5 would give 0.9 for 0):
// there the mean of the deviations is found too and taken from them (8192 x 4096 bf16 22.9
// us, 25.1 where all rows are so; done for every row, it took 8 % at 2048 x 16384 and
// 20000 x 777).  y comes from the sum before its rounding.  Rows of up to 16384 live in
// the registers of one wave or one workgroup, the choice by N; longer ones are read once
// per pass (4096 x 28672 bf16: 141 us, 470 MB in 91 at the rate of a copy).
#include "philox.hpp"
#include "rows.hpp"

namespace coalesce {
namespace {

// Columns n .. n + 7 of the sum (or of the input itself).
template <typename T, typename TS>
struct Input {
  Row<TS> s;
  Row<T> x;
  bool sum;
  __device__ __forceinline__ Input(const NormParams& p, int64_t row)
      : s(p.R ? Row<TS>::in(p.R, p.ldr, row, p.N) : Row<TS>::in(p.X, p.ldx, row, p.N)),
        x(Row<T>::in(p.X, p.ldx, row, p.N)),
        sum(p.R != nullptr) {}
};

// Whether a mean is so large beside the deviations (ve: their variance and eps) that its
// own rounding counts, or ve so large or small that their squares left fp32.
__device__ __forceinline__ bool far(float mean, float ve) {
  return !(mean * mean <= ve && ve >= 0x1p-80f && ve < __builtin_inff());
}
// What such a row's deviations are multiplied by before they are squared.  Those of a small
// ve are at most the root of N 2^-80, those of a large one at most 2^128: lifted, the sum
// of N < 2^23 squares is below 2^103 and 2^119.
__device__ __forceinline__ float lift_of(float ve) {
  return ve < 0x1p-80f ? 0x1p80f : ve < __builtin_inff() ? 1.0f : 0x1p-80f;
}

// One row per TPR threads, CH times 8 of its columns per thread; THREADS / TPR
// rows per workgroup.  A row of one wave needs no barrier.
template <typename T, typename TS, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(NormParams p) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR, ROWS = THREADS / TPR, WAVES = TPR / 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = block_no() * ROWS + wave / WAVES;
  if (row >= p.M) return;  // (whole workgroups where a row has more than one wave)
  const int t = threadIdx.x % TPR;
  __shared__ float part[4][WAVES];
  const Input<T, TS> in(p, row);
  float v[CH][8];
  {
    Raw8<TS> raw[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) raw[c] = in.s.load((c * TPR + t) * 8);
    if (in.sum) {
      Raw8<T> branch[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) branch[c] = in.x.load((c * TPR + t) * 8);
      const DropKey key = drop_key(p.drop);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int n = (c * TPR + t) * 8;
        float b[8];
        Row<T>::widen(branch[c], n, p.N, b);
        Row<TS>::widen(raw[c], n, p.N, v[c]);
        if (p.drop.on) drop8(key, (uint32_t)row, (uint32_t)n, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] += b[e];
      }
      if (p.S) {
        const Row<TS> out = Row<TS>::out(p.S, p.lds, row, p.N);
#pragma unroll
        for (int c = 0; c < CH; ++c) out.store((c * TPR + t) * 8, v[c], (TS*)p.S + row * p.lds);
      }
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c) Row<TS>::widen(raw[c], (c * TPR + t) * 8, p.N, v[c]);
    }
  }
  auto total = [&](float x, int slot) {
    x = wave_sum(x);
    if constexpr (WAVES > 1) {
      if ((threadIdx.x & 63) == 0) part[slot][wave] = x;
      __syncthreads();
      x = part[slot][0];
#pragma unroll
      for (int i = 1; i < WAVES; ++i) x += part[slot][i];
    }
    return x;
  };
  const float count = (float)p.N;  // (divided by, so that a row of one value has that mean)
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += v[c][e];
  float mean = total(sum, 0) / count;
  float sq = 0.0f;
  const bool whole = p.N == TPR * CH * 8;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float d = v[c][e] - mean;
      if (!whole && (c * TPR + t) * 8 + e >= p.N) d = 0.0f;
      v[c][e] = d;
      sq = __builtin_fmaf(d, d, sq);
    }
  float ve = total(sq, 1) / count + p.eps, lift = 1.0f;
  if (far(mean, ve)) {
    lift = lift_of(ve);
    sum = sq = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[c][e] *= lift;
        sum += v[c][e];
      }
    const float off = total(sum, 2) / count;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[c][e] = (c * TPR + t) * 8 + e < p.N ? v[c][e] - off : 0.0f;
        sq = __builtin_fmaf(v[c][e], v[c][e], sq);
      }
    ve = total(sq, 3) / count + p.eps * lift * lift;
    mean += off / lift;
  }
  const float rstd = 1.0f / __builtin_sqrtf(ve);  // of v
  const Row<T> out = Row<T>::out(p.Y, p.ldy, row, p.N);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int n = (c * TPR + t) * 8;
    float w[8], b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.0f, b[e] = 0.0f;
    if (p.weight) read_vec<T>(p.weight, p.wt == DT_F32, n, p.N, w);
    if (p.bias) read_vec<T>(p.bias, p.wt == DT_F32, n, p.N, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[c][e] = __builtin_fmaf(v[c][e] * rstd, w[e], b[e]);
    out.store(n, v[c], (T*)p.Y + row * p.ldy);
  }
  if (t == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd * lift;
  }
}

// Rows longer than the registers: one workgroup per row, three passes
// (five of a row far from zero).  Each
// thread meets the same columns in every pass and writes them in the last, so the
// sum may be formed in place.
template <typename T, typename TS>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormParams p) {
  __shared__ float part[4][16];
  const int64_t row = block_no();
  if (row >= p.M) return;
  const Input<T, TS> in(p, row);
  const DropKey key = drop_key(p.drop);
  auto read = [&](int n, float (&v)[8]) {
    in.s.read(n, v);
    if (!in.sum) return;
    float b[8];
    in.x.read(n, b);
    if (p.drop.on) drop8(key, (uint32_t)row, (uint32_t)n, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += b[e];
  };
  auto total = [&](float x, int slot) {
    x = wave_sum(x);
    if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = x;
    __syncthreads();
    x = part[slot][0];
#pragma unroll
    for (int i = 1; i < 16; ++i) x += part[slot][i];
    return x;
  };
  const float count = (float)p.N;  // (divided by, so that a row of one value has that mean)
  float sum = 0.0f, sq = 0.0f;
  for (int n = threadIdx.x * 8; n < p.N; n += 8192) {
    float v[8];
    read(n, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += v[e];
  }
  const float mean = total(sum, 0) / count;
  float off = 0.0f, lift = 1.0f;  // what is taken from the lifted deviations
  for (int n = threadIdx.x * 8; n < p.N; n += 8192) {
    float v[8];
    read(n, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = n + e < p.N ? v[e] - mean : 0.0f;
      sq = __builtin_fmaf(d, d, sq);
    }
  }
  float ve = total(sq, 1) / count + p.eps;
  if (far(mean, ve)) {
    lift = lift_of(ve);
    sum = sq = 0.0f;
    for (int n = threadIdx.x * 8; n < p.N; n += 8192) {
      float v[8];
      read(n, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += n + e < p.N ? (v[e] - mean) * lift : 0.0f;
    }
    off = total(sum, 2) / count;
    for (int n = threadIdx.x * 8; n < p.N; n += 8192) {
      float v[8];
      read(n, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = n + e < p.N ? (v[e] - mean) * lift - off : 0.0f;
        sq = __builtin_fmaf(d, d, sq);
      }
    }
    ve = total(sq, 3) / count + p.eps * lift * lift;
  }
  const float rstd = 1.0f / __builtin_sqrtf(ve);
  const Row<T> out = Row<T>::out(p.Y, p.ldy, row, p.N);
  for (int n = threadIdx.x * 8; n < p.N; n += 8192) {
    float v[8], w[8], b[8];
    read(n, v);
    if (p.S) Row<TS>::out(p.S, p.lds, row, p.N).store(n, v, (TS*)p.S + row * p.lds);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.0f, b[e] = 0.0f;
    if (p.weight) read_vec<T>(p.weight, p.wt == DT_F32, n, p.N, w);
    if (p.bias) read_vec<T>(p.bias, p.wt == DT_F32, n, p.N, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(((v[e] - mean) * lift - off) * rstd, w[e], b[e]);
    out.store(n, v, (T*)p.Y + row * p.ldy);
  }
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean + off / lift;
    if (p.rstd) p.rstd[row] = rstd * lift;
  }
}

template <typename T, typename TS>
hipError_t norm_typed(const NormParams& p, hipStream_t stream) {
#define COALESCE_NORM(TPR, CH)                                                                                       \
  hipLaunchKernelGGL((norm_kernel<T, TS, TPR, CH>),                                                                  \
                     blocks_grid(TPR < 256 ? ((int64_t)p.M + 256 / TPR - 1) / (256 / TPR) : p.M),                     \
                     dim3(TPR < 256 ? 256 : TPR), 0, stream, p)
  if (p.N <= 512)
    COALESCE_NORM(64, 1);
  else if (p.N <= 1024)
    COALESCE_NORM(64, 2);
  else if (p.N <= 2048)
    COALESCE_NORM(256, 1);
  else if (p.N <= 4096)
    COALESCE_NORM(256, 2);
  else if (p.N <= 8192)
    COALESCE_NORM(512, 2);
  else if (p.N <= 16384)
    COALESCE_NORM(1024, 2);
  else
    hipLaunchKernelGGL((norm_long_kernel<T, TS>), blocks_grid(p.M), dim3(1024), 0, stream, p);
#undef COALESCE_NORM
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormParams& p, DType operand, DType stream_type, hipStream_t stream) {
  if (operand == DT_F32) return norm_typed<float, float>(p, stream);
  if (operand == DT_BF16)
    return stream_type == DT_F32 ? norm_typed<__bf16, float>(p, stream) : norm_typed<__bf16, __bf16>(p, stream);
  return stream_type == DT_F32 ? norm_typed<_Float16, float>(p, stream) : norm_typed<_Float16, _Float16>(p, stream);
}

}  // namespace coalesce
