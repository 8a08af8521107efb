// Quantisation to 8-bit integers on gfx950, symmetric, one scale per row (a token of
// activations) or per column (a channel of weights):
//   scale = amax / 127;  q = rint(x (127 / amax))
// each operation rounded to fp32 by itself, so q is one value and not a matter of
// the kernel's form.  Bound by memory: each row is read once, its 16-bit values stay in
// registers while their largest magnitude is found.  A row of zeros has scale 0.  A
// row that holds an infinity or a NaN has scale NaN and q = 0, so what is computed
// from it is NaN and not a number that looks right.
#include "block.hpp"
#include "rows.hpp"

namespace coalesce {
namespace {

// Magnitudes as integers: they order as the values do, infinities and then NaN above.
__device__ __forceinline__ uint32_t magnitude(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }

struct Scale {
  float scale, inv, lift;
};
// 127 / amax overflows for amax below 2^-121: such rows are lifted by 2^64 first
// (exact), amax with them.
__device__ __forceinline__ Scale scale_of(uint32_t bits) {
  Scale s{0.0f, 0.0f, 1.0f};
  if (bits >= 0x7f800000u) {
    s.scale = __builtin_nanf("");
    s.lift = 0.0f;
  } else if (bits) {
    float a = __builtin_bit_cast(float, bits);
    s.scale = a / 127.0f;
    if (a < 0x1p-100f) s.lift = 0x1p64f;
    s.inv = 127.0f / (a * s.lift);
  }
  return s;
}
__device__ __forceinline__ int quant(float v, const Scale& s) {
  // (rows without a scale give 0, whatever they hold)
  return s.inv == 0.0f ? 0 : (int)__builtin_rintf(v * s.lift * s.inv);
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return (uint32_t)(a & 0xff) | (uint32_t)(b & 0xff) << 8 | (uint32_t)(c & 0xff) << 16 | (uint32_t)d << 24;
}

// 8 values of columns n.. as bytes; `valid` of them lie in the row.
__device__ __forceinline__ void store_q(int8_t* q, int n, int valid, const float (&v)[8], const Scale& s) {
  int i[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) i[e] = quant(v[e], s);
  if (valid >= 8) {
    *(u32x2*)(q + n) = (u32x2){pack4(i[0], i[1], i[2], i[3]), pack4(i[4], i[5], i[6], i[7])};
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < valid) q[n + e] = (int8_t)i[e];
  }
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
  return v;
}

// One row per TPR threads, CH times 8 of its columns per thread.
template <typename T, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void quant_rows_kernel(QuantParams p) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR, ROWS = THREADS / TPR, WAVES = TPR / 64;
  __shared__ uint32_t part[WAVES];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = block_no() * ROWS + wave / WAVES;
  if (row >= p.M) return;
  const int t = threadIdx.x % TPR;
  const Row<T> in = Row<T>::in(p.X, p.ldx, row, p.N);
  Raw8<T> raw[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) raw[c] = in.load((c * TPR + t) * 8);
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float v[8];
    Row<T>::widen(raw[c], (c * TPR + t) * 8, p.N, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, magnitude(v[e]));
  }
  top = wave_max(top);
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) part[wave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WAVES; ++i) top = max(top, part[i]);
  }
  const Scale s = scale_of(top);
  int8_t* q = p.Q + row * p.ldq;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int n = (c * TPR + t) * 8;
    float v[8];
    Row<T>::widen(raw[c], n, p.N, v);
    store_q(q, n, p.N - n, v, s);
  }
  if (t == 0) p.scale[row] = s.scale;
}

// Rows longer than the registers: read twice.
template <typename T>
__global__ __launch_bounds__(1024) void quant_long_kernel(QuantParams p) {
  __shared__ uint32_t part[16];
  const int64_t row = block_no();
  if (row >= p.M) return;
  const Row<T> in = Row<T>::in(p.X, p.ldx, row, p.N);
  uint32_t top = 0;
  for (int n = threadIdx.x * 8; n < p.N; n += 8192) {
    float v[8];
    in.read(n, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, magnitude(v[e]));
  }
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, part[i]);
  const Scale s = scale_of(top);
  for (int n = threadIdx.x * 8; n < p.N; n += 8192) {
    float v[8];
    in.read(n, v);
    store_q(p.Q + row * p.ldq, n, p.N - n, v, s);
  }
  if (threadIdx.x == 0) p.scale[row] = s.scale;
}

// Columns, in four small launches: largest magnitudes set to 0; their maximum over
// ranges of rows, kept as integers in the place of the scales (an integer maximum is
// the same in any order); the values, turned over 64 x 64 at a time in LDS so that rows
// of Q are written in whole 64-byte pieces; and the scales.  Weights go through it once.
__global__ __launch_bounds__(256) void columns_zero_kernel(QuantParams p) {
  const int n = (int)blockIdx.x * 256 + (int)threadIdx.x;
  if (n < p.N) ((uint32_t*)p.scale)[n] = 0u;
}

constexpr int kTopRows = 512;  // rows of a range
template <typename T>
__global__ __launch_bounds__(256) void columns_top_kernel(QuantParams p, int col_blocks) {
  __shared__ uint32_t tops[4][64];
  const int c = threadIdx.x & 63, r = threadIdx.x >> 6;
  const uint32_t no = (uint32_t)block_no(), band = no / (uint32_t)col_blocks;  // (2^41 elements: 2^30 blocks)
  const int n = (int)(no - band * (uint32_t)col_blocks) * 64 + c;
  const int64_t m0 = (int64_t)band * kTopRows;
  const int rows = (int)min((int64_t)kTopRows, (int64_t)p.M - m0);
  uint32_t top = 0;
  if (n < p.N) {
    const T* x = (const T*)p.X + m0 * p.ldx + n;
    for (int m = r; m < rows; m += 32) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (m + 4 * u < rows) top = max(top, magnitude((float)x[(int64_t)(m + 4 * u) * p.ldx]));
    }
  }
  tops[r][c] = top;
  __syncthreads();
  if (r == 0 && n < p.N) {
#pragma unroll
    for (int i = 1; i < 4; ++i) top = max(top, tops[i][c]);
    atomicMax((uint32_t*)p.scale + n, top);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void columns_turn_kernel(QuantParams p, int col_blocks) {
  __shared__ int8_t block[64][64 + 4];
  const int c = threadIdx.x & 63, r = threadIdx.x >> 6;
  const uint32_t no = (uint32_t)block_no(), band = no / (uint32_t)col_blocks;
  const int n0 = (int)(no - band * (uint32_t)col_blocks) * 64, n = n0 + c;
  const int64_t m0 = (int64_t)band * 64;
  const int rows = (int)min((int64_t)64, (int64_t)p.M - m0);
  if (n < p.N) {
    const Scale s = scale_of(((const uint32_t*)p.scale)[n]);
    const T* x = (const T*)p.X + m0 * p.ldx + n;
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      const int m = r + 4 * u;
      if (m < rows) block[c][m] = (int8_t)quant((float)x[(int64_t)m * p.ldx], s);
    }
  }
  __syncthreads();
  // 16 threads of 4 bytes per row of Q
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int row = (threadIdx.x >> 4) + 16 * u, k = (threadIdx.x & 15) * 4;
    if (n0 + row >= p.N) continue;
    int8_t* q = p.Q + (int64_t)(n0 + row) * p.ldq + m0 + k;
    const int valid = rows - k;
    if (valid >= 4) {
      *(uint32_t*)q = *(const uint32_t*)&block[row][k];
    } else {
      for (int e = 0; e < valid; ++e) q[e] = block[row][k + e];
    }
  }
}

__global__ __launch_bounds__(256) void columns_scale_kernel(QuantParams p) {
  const int n = (int)blockIdx.x * 256 + (int)threadIdx.x;
  if (n < p.N) p.scale[n] = scale_of(((const uint32_t*)p.scale)[n]).scale;
}

template <typename T>
hipError_t rows_typed(const QuantParams& p, hipStream_t stream) {
#define COALESCE_ROWS(TPR, CH)                                                                                       \
  hipLaunchKernelGGL((quant_rows_kernel<T, TPR, CH>),                                                                \
                     blocks_grid(TPR < 256 ? ((int64_t)p.M + 256 / TPR - 1) / (256 / TPR) : p.M),                     \
                     dim3(TPR < 256 ? 256 : TPR), 0, stream, p)
  if (p.N <= 512)
    COALESCE_ROWS(64, 1);
  else if (p.N <= 1024)
    COALESCE_ROWS(64, 2);
  else if (p.N <= 2048)
    COALESCE_ROWS(256, 1);
  else if (p.N <= 4096)
    COALESCE_ROWS(256, 2);
  else if (p.N <= 8192)
    COALESCE_ROWS(512, 2);
  else if (p.N <= 16384)
    COALESCE_ROWS(1024, 2);
  else
    hipLaunchKernelGGL((quant_long_kernel<T>), blocks_grid(p.M), dim3(1024), 0, stream, p);
#undef COALESCE_ROWS
  return hipGetLastError();
}

template <typename T>
hipError_t columns_typed(const QuantParams& p, hipStream_t stream) {
  const int64_t col_blocks = ((int64_t)p.N + 63) / 64, ranges = ((int64_t)p.M + kTopRows - 1) / kTopRows;
  const dim3 vec((unsigned)(((int64_t)p.N + 255) / 256));
  hipLaunchKernelGGL(columns_zero_kernel, vec, dim3(256), 0, stream, p);
  if (p.M > 0) {
    hipLaunchKernelGGL((columns_top_kernel<T>), blocks_grid(col_blocks * ranges), dim3(256), 0, stream, p,
                       (int)col_blocks);
    hipLaunchKernelGGL((columns_turn_kernel<T>), blocks_grid(col_blocks * (((int64_t)p.M + 63) / 64)), dim3(256), 0,
                       stream, p, (int)col_blocks);
  }
  hipLaunchKernelGGL(columns_scale_kernel, vec, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(const QuantParams& p, DType dt, hipStream_t stream) {
  if (dt == DT_F32) return rows_typed<float>(p, stream);
  return dt == DT_BF16 ? rows_typed<__bf16>(p, stream) : rows_typed<_Float16>(p, stream);
}

hipError_t launch_quantize_columns(const QuantParams& p, DType dt, hipStream_t stream) {
  if (dt == DT_F32) return columns_typed<float>(p, stream);
  return dt == DT_BF16 ? columns_typed<__bf16>(p, stream) : columns_typed<_Float16>(p, stream);
}

}  // namespace coalesce
