// Backward of the layer norm on gfx950, from the stream s and the statistics of
// the forward:
//   g = dY w;  xh = (s - mean) rstd
//   ds = rstd (g - sum(g) / N - xh sum(g xh) / N) + dS       the stream's gradient
//   dbranch = keep(ds) / (1 - p)                             that of the branch added in front
//   dw = sum over rows of dY xh;  db = sum over rows of dY
// One sweep over the rows computes all of it (8192 x 4096 bf16 with dS, dbranch and a
// dropout: 336 MB in 72 us, 4.7 TB/s, and 6 us for the second launch; a copy reaches
// 5.2): workgroups take rows in turn, a
// thread keeps the sums of its columns in registers from row to row while the next
// row's loads are in flight, and writes them once as a partial sum.  A second small
// launch adds the partials in order (no atomics: the same bits every time); a few
// short rows need none.
// Sums and statistics are fp32.  Rows longer than the registers take one kernel per
// row and one per block of columns instead.
#include <algorithm>

#include "philox.hpp"
#include "rows.hpp"

namespace coalesce {
namespace {

// The sums of columns n to n + 3 of a workgroup: a partial result, or, of the only
// workgroup, the gradient of the weight (i = 0) or of the bias.
__device__ __forceinline__ void put_sums(ArgsOf<NormBwdParams> p, int i, int n, f32x4 s) {
  if (n >= p->ldp) return;
  if (!p->alone) {
    *(f32x4*)(p->partial + ((int64_t)i * gridDim.x + blockIdx.x) * p->ldp + n) = s;
    return;
  }
  void* const out = i ? p->dbias : p->dweight;
  if (!out) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (n + e >= p->N) continue;
    if (p->gt == DT_F32)
      ((float*)out)[n + e] = s[e];
    else if (p->gt == DT_BF16)
      ((__bf16*)out)[n + e] = (__bf16)s[e];
    else
      ((_Float16*)out)[n + e] = (_Float16)s[e];
  }
}

// TPR threads per row, CH times 8 columns each; rows of one wave lie four to a
// workgroup, whose waves' sums meet in LDS at the end.
template <typename T, typename TS, int TPR, int CH, int ROWS>
__global__ __launch_bounds__(TPR * ROWS) void norm_bwd_kernel(NormBwdParams) {  // read through the segment
  const ArgsOf<NormBwdParams> k = (ArgsOf<NormBwdParams>)__builtin_amdgcn_kernarg_segment_ptr();
  constexpr int THREADS = TPR * ROWS, WAVES = TPR / 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = wave / WAVES;  // of the workgroup's rows
  const int t = threadIdx.x % TPR;
  __shared__ f32x2 part[2][ROWS][WAVES];
  // The sums of 16 columns do not fit beside a row in the 128 registers that 1024
  // threads have: they lie in LDS, each thread its own (bf16, 2048 x 16384: 86 us with
  // spilled registers, 68 so; 70 with the next row's loads ahead, which spill again).
  constexpr bool IN_LDS = TPR == 1024 && CH == 2;
  __shared__ f32x4 acc[IN_LDS ? 4 * CH : 1][IN_LDS ? TPR : 1];
  const int M = k->M, N = k->N;
  const float inv_n = 1.0f / (float)N;

  // A row past the last one reads nothing (resources without a range).
  struct In {
    Raw8<T> dy[CH];
    Raw8<TS> s[CH], g[CH];
    float mean, rstd;
  };
  auto load = [&](int64_t row, In& in) {
    const auto p = again<NormBwdParams>(k);
    const bool there = row < M;
    const int cols = there ? N : 0;
    if (!there) row = 0;
    const Row<T> dy = Row<T>::in(p->dY, p->ldy, row, cols);
    const Row<TS> s = Row<TS>::in(p->S, p->lds, row, cols);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      in.dy[c] = dy.load((c * TPR + t) * 8);
      in.s[c] = s.load((c * TPR + t) * 8);
    }
    if (p->dS) {
      const Row<TS> g = Row<TS>::in(p->dS, p->ldg, row, cols);
#pragma unroll
      for (int c = 0; c < CH; ++c) in.g[c] = g.load((c * TPR + t) * 8);
    }
    in.mean = there ? p->mean[row] : 0.0f;
    in.rstd = there ? p->rstd[row] : 0.0f;
  };

  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t row0 = (int64_t)blockIdx.x * ROWS;
  // The next row's loads go out before this one's arithmetic, where the registers hold
  // both.
  constexpr bool AHEAD = !IN_LDS;
  In in, nx;
  if constexpr (AHEAD) load(row0 + sub, in);
  // (behind the first row's loads)
  float aw[CH][8], ab[CH][8], w[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const auto p = again<NormBwdParams>(k);
#pragma unroll
    for (int e = 0; e < 8; ++e) aw[c][e] = ab[c][e] = 0.0f, w[c][e] = 1.0f;
    if constexpr (IN_LDS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[4 * c + i][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    if (p->weight) read_vec<T>(p->weight, p->wt == DT_F32, (c * TPR + t) * 8, p->N, w[c]);
  }
  for (int parity = 0; row0 < M; row0 += step, parity ^= 1) {
    const int64_t row = row0 + sub;
    if constexpr (AHEAD)
      load(row0 + step + sub, nx);
    else
      load(row, in);
    float dy[CH][8], xh[CH][8], c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int n = (c * TPR + t) * 8;
      Row<T>::widen(in.dy[c], n, N, dy[c]);
      Row<TS>::widen(in.s[c], n, N, xh[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // past the row's end dY is 0: nothing of it counts
        xh[c][e] = (xh[c][e] - in.mean) * in.rstd;
        const float g = dy[c][e] * w[c][e];
        c1 += g;
        c2 = __builtin_fmaf(g, xh[c][e], c2);
        if constexpr (!IN_LDS) {
          aw[c][e] = __builtin_fmaf(dy[c][e], xh[c][e], aw[c][e]);
          ab[c][e] += dy[c][e];
        }
      }
      if constexpr (IN_LDS) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x4 a = acc[4 * c + h][t], b = acc[4 * c + 2 + h][t];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = __builtin_fmaf(dy[c][4 * h + e], xh[c][4 * h + e], a[e]);
            b[e] += dy[c][4 * h + e];
          }
          acc[4 * c + h][t] = a;
          acc[4 * c + 2 + h][t] = b;
        }
      }
    }
    // But xh there is -mean rstd, and 0 times that is none where it overflows: such a row's
    // sum is taken again without them (the branch takes 0.3 us at 8192 x 4096 bf16, 0.1 at
    // 1537 x 1001; a select per value 1 us of 40 at 20000 x 777).
    if (__builtin_expect(!(__builtin_fabsf(in.mean * in.rstd) < __builtin_inff()), 0)) {
      c2 = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((c * TPR + t) * 8 + e < N) c2 = __builtin_fmaf(dy[c][e] * w[c][e], xh[c][e], c2);
    }
    c1 = wave_sum(c1);
    c2 = wave_sum(c2);
    if constexpr (WAVES > 1) {
      // two places in turn: a wave that is a row ahead writes the other one
      if ((threadIdx.x & 63) == 0) part[parity][sub][wave % WAVES] = (f32x2){c1, c2};
      __syncthreads();
      c1 = part[parity][sub][0][0];
      c2 = part[parity][sub][0][1];
#pragma unroll
      for (int i = 1; i < WAVES; ++i) {
        c1 += part[parity][sub][i][0];
        c2 += part[parity][sub][i][1];
      }
    }
    c1 *= inv_n;
    c2 *= inv_n;
    const auto p = again<NormBwdParams>(k);
    if (row < M && (p->dX || p->dB)) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int n = (c * TPR + t) * 8;
        float g[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 0.0f;
        if (p->dS) Row<TS>::widen(in.g[c], n, N, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = __builtin_fmaf(dy[c][e], w[c][e], -c1);
          g[e] = __builtin_fmaf(in.rstd, __builtin_fmaf(-xh[c][e], c2, d), g[e]);
        }
        if (p->dX) Row<TS>::out(p->dX, p->ldx, row, N).store(n, g, (TS*)p->dX + row * p->ldx);
        if (p->dB) {
          if (p->drop.on) drop8(drop_key(p->drop), (uint32_t)row, (uint32_t)n, g);
          Row<T>::out(p->dB, p->ldb, row, N).store(n, g, (T*)p->dB + row * p->ldb);
        }
      }
    }
    if constexpr (AHEAD) in = nx;
  }

  const auto p = again<NormBwdParams>(k);
  if (!p->dweight && !p->dbias) return;
  // partial[0]: dw, partial[1]: db, a row of ldp per workgroup
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (ROWS > 1) {
      __shared__ f32x4 meet[ROWS][2 * CH][TPR];
      __syncthreads();
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float(&a)[8] = i ? ab[c] : aw[c];
          meet[sub][2 * c + h][t] = (f32x4){a[4 * h], a[4 * h + 1], a[4 * h + 2], a[4 * h + 3]};
        }
      __syncthreads();
      for (int u = threadIdx.x; u < 2 * CH * TPR; u += THREADS) {
        const int q = u / TPR, l = u % TPR, n = ((q >> 1) * TPR + l) * 8 + 4 * (q & 1);
        f32x4 s = meet[0][q][l];
#pragma unroll
        for (int r = 1; r < ROWS; ++r) s += meet[r][q][l];
        put_sums(p, i, n, s);
      }
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = (c * TPR + t) * 8 + 4 * h;
          const float(&a)[8] = i ? ab[c] : aw[c];
          if constexpr (IN_LDS)
            put_sums(p, i, n, acc[4 * c + 2 * i + h][t]);
          else
            put_sums(p, i, n, (f32x4){a[4 * h], a[4 * h + 1], a[4 * h + 2], a[4 * h + 3]});
        }
    }
  }
}

// Rows longer than the registers: one workgroup per row, two passes.
template <typename T, typename TS>
__global__ __launch_bounds__(1024) void norm_bwd_long_kernel(NormBwdParams p) {
  __shared__ f32x2 part[16];
  const int64_t row = block_no();
  if (row >= p.M) return;
  const Row<T> dyr = Row<T>::in(p.dY, p.ldy, row, p.N);
  const Row<TS> sr = Row<TS>::in(p.S, p.lds, row, p.N);
  const float mean = p.mean[row], rstd = p.rstd[row];
  const DropKey key = drop_key(p.drop);
  auto read = [&](int n, float (&g)[8], float (&xh)[8]) {
    float w[8];
    dyr.read(n, g);
    sr.read(n, xh);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    if (p.weight) read_vec<T>(p.weight, p.wt == DT_F32, n, p.N, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      g[e] *= w[e];
      xh[e] = n + e < p.N ? (xh[e] - mean) * rstd : 0.0f;  // (-mean rstd may be infinite past the end)
    }
  };
  float c1 = 0.0f, c2 = 0.0f;
  for (int n = threadIdx.x * 8; n < p.N; n += 8192) {
    float g[8], xh[8];
    read(n, g, xh);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c1 += g[e];
      c2 = __builtin_fmaf(g[e], xh[e], c2);
    }
  }
  c1 = wave_sum(c1);
  c2 = wave_sum(c2);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = (f32x2){c1, c2};
  __syncthreads();
  c1 = c2 = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    c1 += part[i][0];
    c2 += part[i][1];
  }
  const float inv_n = 1.0f / (float)p.N;
  c1 *= inv_n;
  c2 *= inv_n;
  for (int n = threadIdx.x * 8; n < p.N; n += 8192) {
    float g[8], xh[8], s[8];
    read(n, g, xh);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.0f;
    if (p.dS) Row<TS>::in(p.dS, p.ldg, row, p.N).read(n, s);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = __builtin_fmaf(rstd, __builtin_fmaf(-xh[e], c2, g[e] - c1), s[e]);
    if (p.dX) Row<TS>::out(p.dX, p.ldx, row, p.N).store(n, g, (TS*)p.dX + row * p.ldx);
    if (p.dB) {
      if (p.drop.on) drop8(key, (uint32_t)row, (uint32_t)n, g);
      Row<T>::out(p.dB, p.ldb, row, p.N).store(n, g, (T*)p.dB + row * p.ldb);
    }
  }
}

// Their column sums: 256 columns per workgroup, eight row lanes, a range of rows.
template <typename T, typename TS>
__global__ __launch_bounds__(256) void norm_cols_kernel(NormBwdParams p) {
  __shared__ float meet[8][256];
  const int l = threadIdx.x & 31, lane = threadIdx.x >> 5;
  const int n = (int)blockIdx.x * 256 + l * 8;
  const int64_t first = (int64_t)p.M * blockIdx.y / p.groups, last = (int64_t)p.M * (blockIdx.y + 1) / p.groups;
  float aw[8], ab[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) aw[e] = ab[e] = 0.0f;
  for (int64_t r0 = first; r0 < last; r0 += 8) {
    const int64_t row = r0 + lane;
    if (row >= last) break;
    float dy[8], s[8];
    const T* dp = (const T*)p.dY + row * p.ldy + n;
    const TS* sp = (const TS*)p.S + row * p.lds + n;
    const float mean = p.mean[row], rstd = p.rstd[row];
    if (n + 8 <= p.N) {
      typedef T t8 __attribute__((ext_vector_type(8)));
      typedef TS s8 __attribute__((ext_vector_type(8)));
      const t8 a = *(const t8*)dp;
      const s8 b = *(const s8*)sp;
#pragma unroll
      for (int e = 0; e < 8; ++e) dy[e] = (float)a[e], s[e] = (float)b[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool in = n + e < p.N;
        dy[e] = in ? (float)dp[e] : 0.0f;
        s[e] = in ? (float)sp[e] : mean;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      aw[e] = __builtin_fmaf(dy[e], (s[e] - mean) * rstd, aw[e]);
      ab[e] += dy[e];
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) meet[lane][l * 8 + e] = k ? ab[e] : aw[e];
    __syncthreads();
    const int col = threadIdx.x, at = (int)blockIdx.x * 256 + col;
    float s = meet[0][col];
#pragma unroll
    for (int r = 1; r < 8; ++r) s += meet[r][col];
    if (at < p.ldp) p.partial[((int64_t)k * p.groups + blockIdx.y) * p.ldp + at] = s;
  }
}

// dw and db from the partial sums: 32 columns per workgroup (eight quads, 128 bytes of
// a partial), 64 lanes that take the partials in turn and are added in order.
template <typename TG>
__global__ __launch_bounds__(512) void norm_sums_kernel(NormBwdParams p) {
  __shared__ f32x4 meet[64][8];
  __shared__ float part[16][32];
  TG* const out = (TG*)(blockIdx.y ? p.dbias : p.dweight);
  if (!out) return;
  const int q = threadIdx.x & 7, lane = threadIdx.x >> 3;
  const int n = (int)blockIdx.x * 32 + q * 4;
  const float* src = p.partial + (int64_t)blockIdx.y * p.groups * p.ldp + n;
  f32x4 s = (f32x4){0.f, 0.f, 0.f, 0.f};
  if (n < p.ldp) {
    for (int g = lane; g < p.groups; g += 512) {
      f32x4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = g + 64 * u < p.groups ? *(const f32x4*)(src + (int64_t)(g + 64 * u) * p.ldp)
                                     : (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
  }
  meet[lane][q] = s;
  __syncthreads();
  const int c = threadIdx.x & 31, j = threadIdx.x >> 5;
  float a = 0.0f;
#pragma unroll
  for (int r = 0; r < 4; ++r) a += meet[4 * j + r][c >> 2][c & 3];
  part[j][c] = a;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  a = 0.0f;
#pragma unroll
  for (int r = 0; r < 16; ++r) a += part[r][c];
  const int at = (int)blockIdx.x * 32 + c;
  if (at < p.N) out[at] = (TG)a;
}

constexpr int kLongRow = 16384;

// Partial sums per column: of the workgroups of the sweep, or of the ranges of rows
// of a long one.
struct SumsPlan {
  int groups, ldp;
  bool alone;
};
SumsPlan sums_plan(int64_t M, int64_t N, int num_cus) {
  SumsPlan s{};
  s.ldp = (int)((N + 7) / 8 * 8);
  if (N > kLongRow) {
    s.groups = (int)std::min<int64_t>((M + 63) / 64, 64);
    return s;
  }
  // As many workgroups as a compute unit holds at once; more would run in a second
  // round and write more partials (bf16, 8192 x 4096: 102 us with one, 77 with two, 72
  // with three, 82 with four; 8, 24 and 33 MB of partials), fewer leave it idle.
  const int64_t rows = N <= 1024 ? 4 : 1;
  const int64_t per_cu = N <= 4096 ? 3 : 1;
  s.groups = (int)std::min<int64_t>((M + rows - 1) / rows, num_cus * per_cu);
  // Few short rows are one workgroup's, which writes the gradients itself (8 x 512 bf16:
  // 5.0 us and one launch, 5.7 and two; but 16 x 512 6.8 and 5.7, 2 x 2048 5.9 and 5.8, 1 x
  // 4096 7.3 and 6.7).
  s.alone = M > 0 && (N <= 1024 ? M <= 8 : N <= 2048 && M == 1);
  if (s.alone) s.groups = 1;
  return s;
}

template <typename T, typename TS>
hipError_t bwd_typed(NormBwdParams p, hipStream_t stream, int num_cus) {
  const SumsPlan plan = sums_plan(p.M, p.N, num_cus);
  p.groups = plan.groups;
  p.alone = plan.alone;
  // fp32 streams take more registers: two workgroups of 16 columns per thread fit a
  // compute unit, and a third would run by itself
  const bool wide = (p.N > 512 && p.N <= 1024) || (p.N > 2048 && p.N <= 4096);
  if (sizeof(TS) == 4 && wide) p.groups = std::min(p.groups, 2 * num_cus);
  p.ldp = plan.ldp;
  const bool sums = p.dweight || p.dbias;
  if (p.M > 0) {
#define COALESCE_NORM(TPR, CH, ROWS) \
  hipLaunchKernelGGL((norm_bwd_kernel<T, TS, TPR, CH, ROWS>), dim3(p.groups), dim3(TPR * ROWS), 0, stream, p)
    if (p.N <= 512)
      COALESCE_NORM(64, 1, 4);
    else if (p.N <= 1024)
      COALESCE_NORM(64, 2, 4);
    else if (p.N <= 2048)
      COALESCE_NORM(256, 1, 1);
    else if (p.N <= 4096)
      COALESCE_NORM(256, 2, 1);
    else if (p.N <= 8192)
      COALESCE_NORM(1024, 1, 1);
    else if (p.N <= kLongRow)
      COALESCE_NORM(1024, 2, 1);
    else {
      if (p.dX || p.dB)
        hipLaunchKernelGGL((norm_bwd_long_kernel<T, TS>), blocks_grid(p.M), dim3(1024), 0, stream, p);
      if (sums)
        hipLaunchKernelGGL((norm_cols_kernel<T, TS>), dim3((unsigned)((p.ldp + 255) / 256), p.groups), dim3(256), 0,
                           stream, p);
    }
#undef COALESCE_NORM
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !sums) return e;
  }
  if (!sums || p.alone) return hipSuccess;
  const dim3 grid((unsigned)((p.N + 31) / 32), 2);
  if (p.gt == DT_F32)
    hipLaunchKernelGGL((norm_sums_kernel<float>), grid, dim3(512), 0, stream, p);
  else if (p.gt == DT_BF16)
    hipLaunchKernelGGL((norm_sums_kernel<__bf16>), grid, dim3(512), 0, stream, p);
  else
    hipLaunchKernelGGL((norm_sums_kernel<_Float16>), grid, dim3(512), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

size_t norm_backward_workspace(int64_t M, int64_t N, int num_cus) {
  const SumsPlan plan = sums_plan(M, N, num_cus);
  return (size_t)plan.groups * (size_t)plan.ldp * 8;
}

hipError_t launch_norm_backward(NormBwdParams p, DType operand, DType stream_type, hipStream_t stream, int num_cus) {
  if (operand == DT_F32) return bwd_typed<float, float>(p, stream, num_cus);
  if (operand == DT_BF16)
    return stream_type == DT_F32 ? bwd_typed<__bf16, float>(p, stream, num_cus)
                                 : bwd_typed<__bf16, __bf16>(p, stream, num_cus);
  return stream_type == DT_F32 ? bwd_typed<_Float16, float>(p, stream, num_cus)
                               : bwd_typed<_Float16, _Float16>(p, stream, num_cus);
}

}  // namespace coalesce
