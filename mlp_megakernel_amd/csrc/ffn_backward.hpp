// Backward of the feed-forward operators:
//   gated product       dZu = dY act(Zg),  dZg = dY Zu act'(Zg)
//   GEMM with residual  dZ  = dY act'(Z)   (and dR = dY, nothing to compute)
//   dX = sum_i dZi Wi^T,  dWi = X^T dZi,  dbi[n] = sum_m dZi[m][n]
// One elementwise pass turns the stored pre-activations and the arriving
// gradient into the dZi, rounded once to the input type because they are the
// matrix products' operands, and sums their columns in fp32 before that
// rounding.  The rounding adds its half step to that of the result (bf16: 0.0023
// of a gradient's norm against 0.0017, fp16 0.00029 against 0.00021), and in
// fp16 the range ends at 65504 and 2^-24; two operands per value (high and low
// part) would avoid both at twice the matrix work.  Both dZi Wi^T run as one K loop over two segments, both X^T dZi
// as one launch whose tiles share X.
#pragma once
#include "ffn_plan.hpp"
#include "gemm16_core.hpp"

namespace coalesce {
namespace {

// Eight consecutive elements, whole (16-byte accesses) or `valid` of them.
template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    const f32x4 a = *(const f32x4*)src, b = *(const f32x4*)(src + 4);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      f[r] = a[r];
      f[4 + r] = b[r];
    }
  } else {
    typedef T t8 __attribute__((ext_vector_type(8)));
    const t8 a = *(const t8*)src;
#pragma unroll
    for (int r = 0; r < 8; ++r) f[r] = (float)a[r];
  }
}
template <typename T>
__device__ __forceinline__ void load8(const T* src, int valid, float (&f)[8]) {
  for (int r = 0; r < 8; ++r) f[r] = r < valid ? (float)src[r] : 0.0f;
}
template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&f)[8]) {
  typedef T t8 __attribute__((ext_vector_type(8)));
  t8 a;
#pragma unroll
  for (int r = 0; r < 8; ++r) a[r] = (T)f[r];
  *(t8*)dst = a;
}

// dZ of eight columns of one row, added to the column sums.
template <int ACT, bool GATED>
__device__ __forceinline__ void dz8(const float (&dy)[8], const float (&zg)[8], const float (&zu)[8], float (&dg)[8],
                                    float (&du)[8], float (&sg)[8], float (&su)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f = 0.0f, d = 1.0f;
    if (ACT != ACT_NONE || GATED) act_and_grad<ACT>(zg[i], f, d);
    dg[i] = GATED ? dy[i] * zu[i] * d : dy[i] * d;
    du[i] = dy[i] * f;
    sg[i] += dg[i];
    su[i] += du[i];
  }
}

// Workgroup (column block, row chunk); partial column sums of dZi to
// sums[(chunk * 2 + i) * N + n].  A thread takes eight columns of R rows at a
// time, all their loads (16 bytes each) in flight before the first use; the
// chunk's and the matrix' ends go row by row and element by element.  Whole and
// ragged column blocks are apart, so that no test of `valid` stands between a
// load and the next: with the tests in one loop, 8192 x 16384 of a gated bf16
// product took 314 us; now 236 us for 0.8 GB read and 0.5 GB written (5.6 TB/s,
// above a large copy's 5.1), and 1537 x 2731 in fp16 15.6 us instead of 20.
template <typename T, typename TD, int ACT, bool GATED>
__global__ __launch_bounds__(256) void dz_kernel(DzParams p) {
  constexpr bool NEEDS_Z = ACT != ACT_NONE || GATED;
  constexpr int R = 2;
  const int c = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int n = blockIdx.x * DZ_COLS + c * 8;
  const int64_t r0 = (int64_t)blockIdx.y * p.chunk_rows, r1 = min(r0 + p.chunk_rows, (int64_t)p.M);
  const TD* dY = (const TD*)p.dY + n;
  const T* Zg = (const T*)p.Z[0] + n;
  const T* Zu = (const T*)p.Z[1] + n;
  T* Dg = p.dZ[0] ? (T*)p.dZ[0] + n : nullptr;
  T* Du = GATED && p.dZ[1] ? (T*)p.dZ[1] + n : nullptr;
  float sg[8], su[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sg[i] = su[i] = 0.0f;
  const int valid = min(8, p.N - n);
  int64_t m = r0 + rl;
  if (valid == 8) {
    for (; m + (R - 1) * DZ_ROWS < r1; m += R * DZ_ROWS) {
      float dy[R][8], zg[R][8], zu[R][8], dg[8], du[8];
#pragma unroll
      for (int h = 0; h < R; ++h) {
        load8<TD>(dY + (m + h * DZ_ROWS) * p.ldd, dy[h]);
        if (NEEDS_Z) load8<T>(Zg + (m + h * DZ_ROWS) * p.ldz, zg[h]);
        if (GATED) load8<T>(Zu + (m + h * DZ_ROWS) * p.ldz, zu[h]);
      }
#pragma unroll
      for (int h = 0; h < R; ++h) {
        dz8<ACT, GATED>(dy[h], zg[h], zu[h], dg, du, sg, su);
        if (Dg) store8<T>(Dg + (m + h * DZ_ROWS) * p.ldw, dg);
        if (Du) store8<T>(Du + (m + h * DZ_ROWS) * p.ldw, du);
      }
    }
    for (; m < r1; m += DZ_ROWS) {
      float dy[8], zg[8], zu[8], dg[8], du[8];
      load8<TD>(dY + m * p.ldd, dy);
      if (NEEDS_Z) load8<T>(Zg + m * p.ldz, zg);
      if (GATED) load8<T>(Zu + m * p.ldz, zu);
      dz8<ACT, GATED>(dy, zg, zu, dg, du, sg, su);
      if (Dg) store8<T>(Dg + m * p.ldw, dg);
      if (Du) store8<T>(Du + m * p.ldw, du);
    }
  } else if (valid > 0) {
    for (; m < r1; m += DZ_ROWS) {
      float dy[8], zg[8], zu[8], dg[8], du[8];
      load8<TD>(dY + m * p.ldd, valid, dy);
      if (NEEDS_Z) load8<T>(Zg + m * p.ldz, valid, zg);
      if (GATED) load8<T>(Zu + m * p.ldz, valid, zu);
      dz8<ACT, GATED>(dy, zg, zu, dg, du, sg, su);
      for (int i = 0; i < valid; ++i) {
        if (Dg) Dg[m * p.ldw + i] = (T)dg[i];
        if (Du) Du[m * p.ldw + i] = (T)du[i];
      }
    }
  }
  if (!p.sums) return;
  // the 8 row lanes' sums, added in lane order
  __shared__ float part[DZ_ROWS][DZ_COLS + 4];
#pragma unroll
  for (int i = 0; i < (GATED ? 2 : 1); ++i) {
    if (i) __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) part[rl][c * 8 + e] = i ? su[e] : sg[e];
    __syncthreads();
    const int col = blockIdx.x * DZ_COLS + threadIdx.x;
    if (col < p.N) {
      float t = 0.0f;
#pragma unroll
      for (int r = 0; r < DZ_ROWS; ++r) t += part[r][threadIdx.x];
      p.sums[((int64_t)blockIdx.y * 2 + i) * p.N + col] = t;
    }
  }
}

// db_i[n] = the chunks' column sums: 8 groups of threads take every eighth
// chunk, eight loads in flight, and are added in group order.
template <typename TG>
__global__ __launch_bounds__(256) void bias_grad_kernel(const float* sums, int chunks, int N, TG* db0, TG* db1) {
  constexpr int COLS = 32, GROUPS = 8;
  __shared__ float part[GROUPS][COLS];
  const int c = threadIdx.x % COLS, g = threadIdx.x / COLS;
  const int n = blockIdx.x * COLS + c, i = blockIdx.y;
  TG* db = i ? db1 : db0;
  float t = 0.0f;
  if (n < N)
    for (int k = g; k < chunks; k += 8 * GROUPS) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = k + u * GROUPS < chunks ? sums[((int64_t)(k + u * GROUPS) * 2 + i) * N + n] : 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u) t += v[u];
    }
  part[g][c] = t;
  __syncthreads();
  if (g || n >= N || !db) return;
  t = part[0][c];
#pragma unroll
  for (int u = 1; u < GROUPS; ++u) t += part[u][c];
  db[n] = (TG)t;
}

template <typename T, typename TD, bool GATED>
hipError_t dz_act(const DzParams& p, int act, dim3 grid, hipStream_t stream) {
  switch (act) {
    case ACT_GELU: hipLaunchKernelGGL((dz_kernel<T, TD, ACT_GELU, GATED>), grid, dim3(256), 0, stream, p); break;
    case ACT_SOFTPLUS: hipLaunchKernelGGL((dz_kernel<T, TD, ACT_SOFTPLUS, GATED>), grid, dim3(256), 0, stream, p); break;
    case ACT_RELU: hipLaunchKernelGGL((dz_kernel<T, TD, ACT_RELU, GATED>), grid, dim3(256), 0, stream, p); break;
    case ACT_SILU: hipLaunchKernelGGL((dz_kernel<T, TD, ACT_SILU, GATED>), grid, dim3(256), 0, stream, p); break;
    default: hipLaunchKernelGGL((dz_kernel<T, TD, ACT_NONE, GATED>), grid, dim3(256), 0, stream, p); break;
  }
  return hipGetLastError();
}

template <typename T, typename TO, Lay LA, Lay LB, int SEGS>
hipError_t store_tiles(const TileOp& o, int variant, hipStream_t stream, int num_cus) {
#define COALESCE_TILE(...) launch_tile<T, TO, LA, LB, SEGS, EPI_STORE, TileGeo<__VA_ARGS__>>(o, stream, num_cus)
  if constexpr (LA == LAY_K) {
    switch (variant) {
      case kShape224: return COALESCE_TILE(224, 256, 8, 2, 1, 1);
      case kShape192: return COALESCE_TILE(192, 256, 8, 2, 1, 1);
      case kShape160: return COALESCE_TILE(160, 256, 8, 2, 1, 1, 3);
    }
  }
  switch (variant) {
    case kShape256: return COALESCE_TILE(256, 256, 8, 2, 1, 1);
    case kShape128: return COALESCE_TILE(128, 128, 4, 2, 2, 1);
    case kShape128Deep: return COALESCE_TILE(128, 128, 4, 2, 1, 1, 3);
    case kShape64Deep: return COALESCE_TILE(64, 64, 4, 2, 3, 1, 3);
    default: return COALESCE_TILE(64, 64, 4, 2, 4, 1);
  }
#undef COALESCE_TILE
}

// One of the backward's products: stored directly, or split into fp32 partial
// results that the combining pass sums.
template <typename T, typename TO, Lay LA, Lay LB, int SEGS>
hipError_t product(TileOp o, const TilePlan& plan, DType out, hipStream_t stream, int num_cus, float* ws) {
  o.splits = plan.splits;
  if (plan.splits <= 1) return store_tiles<T, TO, LA, LB, SEGS>(o, plan.variant, stream, num_cus);
  CombineOp c{};
  c.ldp = partial_pitch(o.N);
  c.split_stride = (int64_t)o.M * c.ldp;
  c.splits = o.splits;
  c.products = o.batch;
  const size_t one = align256((size_t)o.splits * (size_t)c.split_stride * 4) / 4;
  for (int i = 0; i < o.batch; ++i) {
    c.P[i] = ws + i * one;
    c.Y[i] = o.Y[i];
    o.Y[i] = (void*)c.P[i];
  }
  c.ldy = o.ldy;
  c.M = o.M;
  c.N = o.N;
  o.ldy = c.ldp;
  o.split_stride = c.split_stride;
#define COALESCE_TILE(...) launch_tile<T, float, LA, LB, SEGS, EPI_STORE, TileGeo<__VA_ARGS__>>(o, stream, num_cus)
  const hipError_t e = plan.variant == kShape128       ? COALESCE_TILE(128, 128, 4, 2, 2, 1)
                       : plan.variant == kShape128Deep ? COALESCE_TILE(128, 128, 4, 2, 1, 1, 3)
                                                       : COALESCE_TILE(64, 64, 4, 2, 4, 1);
#undef COALESCE_TILE
  if (e != hipSuccess) return e;
  return launch_combine(c, COMBINE_STORE, out, out, stream, num_cus);
}

template <typename T, typename TG>
hipError_t backward_t(const FfnBwdParams& p, DType in, DType grad, bool gated, bool dy32, int act, hipStream_t stream,
                      int num_cus, char* ws) {
  const BwdPlan b = bwd_plan(p.M, p.N, p.K, gated, num_cus);
  float* const partial = (float*)(ws + b.partial_at);
  const int nw = gated ? 2 : 1;
  const bool want_db = p.db[0] || p.db[1];
  const bool products = p.dX || p.dW[0] || p.dW[1];
  // without an activation dZ is dY itself
  const bool as_is = !gated && act == ACT_NONE && !dy32;
  DzParams d{};
  d.dY = p.dY;
  d.ldd = p.ldd;
  d.Z[0] = p.Z[0];
  d.Z[1] = p.Z[1];
  d.ldz = p.ldz;
  d.dZ[0] = products && !as_is ? ws : nullptr;
  d.dZ[1] = products && gated ? ws + b.dz_bytes : nullptr;
  d.ldw = b.ldw;
  d.sums = want_db ? (float*)(ws + b.sums_at) : nullptr;
  d.M = p.M;
  d.N = p.N;
  d.chunk_rows = b.chunk_rows;
  hipError_t e = hipSuccess;
  if (p.M > 0 && p.N > 0 && (d.dZ[0] || d.sums)) {
    const dim3 grid((unsigned)((p.N + DZ_COLS - 1) / DZ_COLS), (unsigned)b.chunks);
    if (gated)
      e = dy32 ? dz_act<T, float, true>(d, act, grid, stream) : dz_act<T, T, true>(d, act, grid, stream);
    else
      e = dy32 ? dz_act<T, float, false>(d, act, grid, stream) : dz_act<T, T, false>(d, act, grid, stream);
    if (e != hipSuccess) return e;
  }
  if (want_db && p.N > 0) {
    hipLaunchKernelGGL((bias_grad_kernel<TG>), dim3((unsigned)((p.N + 31) / 32), nw), dim3(256), 0, stream,
                       (const float*)(ws + b.sums_at), b.chunks, p.N, (TG*)p.db[0], (TG*)p.db[1]);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const void* dZ[2] = {as_is ? p.dY : (const void*)ws, gated ? (const void*)(ws + b.dz_bytes) : nullptr};
  const int64_t ldw = as_is ? p.ldd : b.ldw;
  if (p.dX && p.M > 0 && p.K > 0) {
    TileOp o{};
    for (int i = 0; i < nw; ++i) {
      o.a[i] = dZ[i];
      o.b[i] = p.W[i];
    }
    o.lda = ldw;
    o.ldb = p.ldw;
    o.M = p.M;
    o.N = p.K;
    o.K = p.N;
    o.batch = 1;
    o.Y[0] = p.dX;
    o.ldy = p.lddx;
    e = gated ? product<T, T, LAY_K, LAY_K, 2>(o, b.dx, in, stream, num_cus, partial)
              : product<T, T, LAY_K, LAY_K, 1>(o, b.dx, in, stream, num_cus, partial);
    if (e != hipSuccess) return e;
  }
  if ((p.dW[0] || p.dW[1]) && p.N > 0 && p.K > 0) {
    TileOp o{};
    o.a[0] = p.X;
    o.lda = p.ldx;
    o.ldb = ldw;
    o.ldy = p.lddw;
    o.M = p.K;
    o.N = p.N;
    o.K = p.M;
    o.batch = 0;
    for (int i = 0; i < nw; ++i)
      if (p.dW[i]) {
        o.b[o.batch] = dZ[i];
        o.Y[o.batch] = p.dW[i];
        ++o.batch;
      }
    e = product<T, TG, LAY_X, LAY_X, 1>(o, b.dw, grad, stream, num_cus, partial);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T>
hipError_t backward_typed(const FfnBwdParams& p, DType in, bool gated, DType dy, DType grad, int act,
                          hipStream_t stream, int num_cus, void* workspace) {
  const bool dy32 = dy == DT_F32;
  if (grad == DT_F32) return backward_t<T, float>(p, in, grad, gated, dy32, act, stream, num_cus, (char*)workspace);
  return backward_t<T, T>(p, in, grad, gated, dy32, act, stream, num_cus, (char*)workspace);
}

}  // namespace
}  // namespace coalesce
