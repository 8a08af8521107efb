// The global norm of a list of gradients, and the list scaled by
//   c = min(1, max_norm / (norm + 1e-6)).
//
// Two sweeps: the first sums squares (or takes the largest magnitude) of every
// tensor of the list into one partial per workgroup, the second adds the
// partials -- every workgroup all of them, in the same order, so no third
// launch -- and scales.  A table has up to 2048 partials, so those reads grow with
// the square of the number of tables: nothing at hundreds of tensors, 2048 x 8
// bytes per workgroup and table, but what would count at tens of thousands.  The list travels in the kernel arguments, a table of
// up to kClipTensors tensors per launch, so nothing is copied to the device and
// the calls can be captured.  Work is cut into chunks of equal size over all
// tensors of a table; workgroup b takes chunks b, b + grid, ...: which element
// meets which partial does not depend on timing, so repeated calls give the
// same bits.  Squares are summed in fp64: they neither overflow nor round
// (an fp32 gradient above 2^64 would overflow an fp32 sum), and at HBM speed
// the conversion and the fma hide behind the loads.
//
// Both sweeps are bound by memory.  The second one goes from the list's end to
// its start, so that it finds the last kKeepBytes, which the first one reads
// through the caches, in the 256 MB one; what lies before them is read past the
// caches (non-temporal), and so are the results of a list above kPastBytes
// written.  1.2 GB of bf16: 705 us with every access through the caches, 647
// past them, 607 with 160 MB kept (the norm alone 214 -> 184 us, 6.5 TB/s); a
// list of 64 MB 38 us past them and 35 through them, of 128 MB 71 and 80.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace coalesce {
namespace {

constexpr int THREADS = 256;
constexpr int64_t kKeepBytes = int64_t(160) << 20, kPastBytes = int64_t(80) << 20;

template <bool PAST, typename V>
__device__ __forceinline__ V load_past(const V* p) {
  if constexpr (PAST)
    return __builtin_nontemporal_load(p);
  else
    return *p;
}
template <bool PAST, typename V>
__device__ __forceinline__ void store_past(V* p, V v) {
  if constexpr (PAST)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}

// x c as fp32, then one rounding to T: kept apart so that every path through
// the kernel rounds alike (a fused multiply and conversion to fp16 rounds once
// where two instructions round twice).
template <typename T>
__device__ __forceinline__ T scaled(T x, float c) {
  float r = (float)x * c;
  asm("" : "+v"(r));
  return (T)r;
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) { return (b > a || b != b) ? b : a; }

template <typename T>
struct Vec {
  static constexpr int N = 16 / (int)sizeof(T);
  typedef T type __attribute__((ext_vector_type(N)));
};

template <bool INF>
struct Accum {
  double s = 0.0;
  float m = 0.0f;
  __device__ __forceinline__ void add(float x) {
    if constexpr (INF) {
      m = max_nan(m, __builtin_fabsf(x));
    } else {
      const double d = (double)x;
      s = __builtin_fma(d, d, s);
    }
  }
};

// A thread's four accumulators together.
template <bool INF>
__device__ __forceinline__ double thread_total(const Accum<INF> (&a)[4]) {
  if constexpr (INF)
    return (double)max_nan(max_nan(a[0].m, a[1].m), max_nan(a[2].m, a[3].m));
  else
    return (a[0].s + a[1].s) + (a[2].s + a[3].s);
}

// The workgroup's total, in thread 0 (and, with the second step, everywhere).
template <bool INF>
__device__ __forceinline__ double block_total(double v) {
  __shared__ double wave_part[THREADS / 64];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const double o = __shfl_xor(v, off);
    v = INF ? (double)max_nan((float)v, (float)o) : v + o;
  }
  if ((threadIdx.x & 63) == 0) wave_part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = wave_part[0];
#pragma unroll
  for (int i = 1; i < THREADS / 64; ++i) v = INF ? (double)max_nan((float)v, (float)wave_part[i]) : v + wave_part[i];
  return v;
}

// The tensor of chunk c of a table.
template <typename Table>
__device__ __forceinline__ int find_tensor(const Table& t, int64_t c) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (c < t.chunk_end[mid])
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// One chunk of n elements at p, added to the four accumulators of thread `tid`
// of the NT that share it.
template <typename T, bool INF, bool PAST, int NT = THREADS>
__device__ __forceinline__ void add_chunk(const T* p, int64_t n, Accum<INF> (&a)[4], int tid) {
  typedef typename Vec<T>::type V;
  constexpr int VN = Vec<T>::N;
  const int64_t head = min(n, (int64_t)(((16 - ((uintptr_t)p & 15)) & 15) / sizeof(T)));
  const V* pv = (const V*)(p + head);
  const int64_t nv = (n - head) / VN;
  if ((int64_t)tid < head) a[0].add((float)p[tid]);
  int64_t k = tid;
  for (; k + 3 * NT < nv; k += 4 * NT) {
    V v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = load_past<PAST>(pv + k + u * NT);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < VN; ++e) a[u].add((float)v[u][e]);
  }
  for (; k < nv; k += NT) {
    const V v = load_past<PAST>(pv + k);
#pragma unroll
    for (int e = 0; e < VN; ++e) a[0].add((float)v[e]);
  }
  const int64_t done = head + nv * VN;
  if ((int64_t)tid < n - done) a[1].add((float)p[done + tid]);
}

template <typename T, bool INF>
__global__ __launch_bounds__(THREADS) void norm_kernel(ClipTable t, double* partial) {
  Accum<INF> a[4];
  const int64_t chunks = t.chunk_end[t.count - 1];
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = find_tensor(t, c);
    const int64_t e0 = (c - (i ? t.chunk_end[i - 1] : 0)) * t.chunk;
    const int64_t n = min(t.numel[i] - e0, t.chunk);
    const T* p = (const T*)t.src[i] + e0;
    if (c < t.keep)
      add_chunk<T, INF, true>(p, n, a, threadIdx.x);
    else
      add_chunk<T, INF, false>(p, n, a, threadIdx.x);
  }
  const double v = block_total<INF>(thread_total(a));
  if (threadIdx.x == 0) partial[blockIdx.x] = v;
}

// Where piece c of a table of matrices lies: `rows` rows from row r0 on,
// elements [c0, c0 + n) of each.  A piece is as many whole rows as `chunk`
// elements hold, or a part of one row that is longer.
struct Piece {
  int64_t r0, rows, c0, n;
};
__device__ __forceinline__ Piece piece_at(const ClipRows& t, int i, int64_t c) {
  const int64_t k = c - (i ? t.chunk_end[i - 1] : 0), cols = t.cols[i], parts = (cols + t.chunk - 1) / t.chunk;
  Piece p;
  if (parts > 1) {
    p.r0 = k / parts;
    p.rows = 1;
    p.c0 = (k - p.r0 * parts) * t.chunk;
    p.n = min(cols - p.c0, t.chunk);
  } else {
    const int64_t per = t.chunk / cols;
    p.r0 = k * per;
    p.rows = min(t.rows[i] - p.r0, per);
    p.c0 = 0;
    p.n = cols;
  }
  return p;
}

// Matrices whose rows lie apart (what stands between the rows is not touched): a
// wave takes a piece, one row after the other.  Bound by memory where a row is
// some hundred bytes or more: norm and scaling of six 2731 x 1001 fp32 gradients,
// 66 MB, 41 us against 34 of dense ones, one of 4096 x 11003 in bf16 48 against 49;
// 100000 rows of 5, a row's latency each, 41 against 14.
template <typename T, bool INF>
__global__ __launch_bounds__(THREADS) void norm_rows_kernel(ClipRows t, double* partial) {
  Accum<INF> a[4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t chunks = t.chunk_end[t.count - 1];
  for (int64_t c = (int64_t)blockIdx.x * (THREADS / 64) + wave; c < chunks; c += (int64_t)gridDim.x * (THREADS / 64)) {
    const int i = find_tensor(t, c);
    const Piece q = piece_at(t, i, c);
    const T* p = (const T*)t.src[i] + q.r0 * t.ld[i] + q.c0;
    for (int64_t r = 0; r < q.rows; ++r) add_chunk<T, INF, false, 64>(p + r * t.ld[i], q.n, a, lane);
  }
  const double v = block_total<INF>(thread_total(a));
  if (threadIdx.x == 0) partial[blockIdx.x] = v;
}

// The norm from all partials, the same value in every thread of every
// workgroup.
template <bool INF>
__device__ __forceinline__ double total_norm(const double* partial, int n) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += THREADS)
    v = INF ? (double)max_nan((float)v, (float)partial[i]) : v + partial[i];
  v = block_total<INF>(v);
  return INF ? v : __builtin_sqrt(v);
}

template <bool INF>
__global__ __launch_bounds__(THREADS) void norm_only_kernel(const double* partial, int n, float* norm) {
  const double v = total_norm<INF>(partial, n);
  if (threadIdx.x == 0) norm[0] = (float)v;
}

// o = p c over n elements, by thread `tid` of NT.
template <typename T, bool PAST, int NT = THREADS>
__device__ __forceinline__ void scale_chunk(const T* p, T* o, int64_t n, float coef, int tid) {
  typedef typename Vec<T>::type V;
  constexpr int VN = Vec<T>::N;
  if ((((uintptr_t)p ^ (uintptr_t)o) & 15) != 0) {  // no common 16-byte grid
    for (int64_t k = tid; k < n; k += NT) o[k] = scaled<T>(p[k], coef);
    return;
  }
  const int64_t head = min(n, (int64_t)(((16 - ((uintptr_t)p & 15)) & 15) / sizeof(T)));
  const V* pv = (const V*)(p + head);
  V* ov = (V*)(o + head);
  const int64_t nv = (n - head) / VN;
  if ((int64_t)tid < head) o[tid] = scaled<T>(p[tid], coef);
  int64_t k = tid;
  for (; k + 3 * NT < nv; k += 4 * NT) {
    V v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = load_past<PAST>(pv + k + u * NT);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
      for (int e = 0; e < VN; ++e) v[u][e] = scaled<T>(v[u][e], coef);
      store_past<PAST>(ov + k + u * NT, v[u]);
    }
  }
  for (; k < nv; k += NT) {
    V v = load_past<PAST>(pv + k);
#pragma unroll
    for (int e = 0; e < VN; ++e) v[e] = scaled<T>(v[e], coef);
    store_past<PAST>(ov + k, v);
  }
  const int64_t done = head + nv * VN;
  if ((int64_t)tid < n - done) o[done + tid] = scaled<T>(p[done + tid], coef);
}

// c = min(1, max_norm / (norm + 1e-6)) in every thread; a NaN stays one.
template <bool INF>
__device__ __forceinline__ float scale_of(const double* partial, int n_partial, double max_norm, float* norm) {
  const double total = total_norm<INF>(partial, n_partial);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = (float)total;
  const double q = max_norm / (total + 1e-6);
  return q < 1.0 || q != q ? (float)q : 1.0f;
}

template <typename T, bool INF>
__global__ __launch_bounds__(THREADS) void scale_kernel(ClipTable t, const double* partial, int n_partial,
                                                        double max_norm, bool past, float* norm) {
  const float coef = scale_of<INF>(partial, n_partial, max_norm, norm);
  for (int64_t c = t.chunk_end[t.count - 1] - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const int i = find_tensor(t, c);
    if (coef == 1.0f && t.src[i] == t.dst[i]) continue;  // in place and nothing to scale
    const int64_t e0 = (c - (i ? t.chunk_end[i - 1] : 0)) * t.chunk;
    const int64_t n = min(t.numel[i] - e0, t.chunk);
    const T* p = (const T*)t.src[i] + e0;
    T* o = (T*)t.dst[i] + e0;
    if (past)
      scale_chunk<T, true>(p, o, n, coef, threadIdx.x);
    else
      scale_chunk<T, false>(p, o, n, coef, threadIdx.x);
  }
}

template <typename T, bool INF>
__global__ __launch_bounds__(THREADS) void scale_rows_kernel(ClipRows t, const double* partial, int n_partial,
                                                             double max_norm, float* norm) {
  const float coef = scale_of<INF>(partial, n_partial, max_norm, norm);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t step = (int64_t)gridDim.x * (THREADS / 64);
  for (int64_t c = t.chunk_end[t.count - 1] - 1 - ((int64_t)blockIdx.x * (THREADS / 64) + wave); c >= 0; c -= step) {
    const int i = find_tensor(t, c);
    if (coef == 1.0f && t.src[i] == t.dst[i]) continue;
    const Piece q = piece_at(t, i, c);
    const T* p = (const T*)t.src[i] + q.r0 * t.ld[i] + q.c0;
    T* o = (T*)t.dst[i] + q.r0 * t.ld_out[i] + q.c0;
    for (int64_t r = 0; r < q.rows; ++r)
      scale_chunk<T, false, 64>(p + r * t.ld[i], o + r * t.ld_out[i], q.n, coef, lane);
  }
}

// Elements per chunk: 64 KB of a large list; of a small one as many as give
// its launch about a workgroup per compute unit, at least 1024.
int64_t chunk_elems(int64_t total, int64_t es, int num_cus) {
  int64_t c = 65536 / es;
  while (c > 1024 && total / c < num_cus) c /= 2;
  return c;
}

int64_t dtype_bytes(int dt) { return dt == DT_F32 ? 4 : 2; }

bool lies_apart(const ClipList& l, int64_t i) { return l.cols && l.cols[i] != 0; }

// Calls fn(table, dtype) for the list's tables of dense tensors: of one dtype,
// empty ones left out, in list order or (`backwards`) the tables from the list's end, each
// in list order within itself.
template <typename F>
hipError_t for_tables(const ClipList& l, int num_cus, bool backwards, F fn) {
  int64_t total = 0, bytes = 0;
  for (int64_t i = 0; i < l.count; ++i) {
    if (lies_apart(l, i)) continue;
    total += l.numel[i];
    bytes += l.numel[i] * dtype_bytes(l.dtype[i]);
  }
  int64_t before = 0;  // bytes of the tables so far
  static const int order[2][3] = {{DT_F32, DT_F16, DT_BF16}, {DT_BF16, DT_F16, DT_F32}};
  for (int dt : order[backwards]) {
    const int64_t es = dtype_bytes(dt), chunk = chunk_elems(total, es, num_cus);
    ClipTable t{};
    t.chunk = chunk;
    for (int64_t k = 0; k <= l.count; ++k) {
      const bool end = k == l.count;
      const int64_t i = backwards ? l.count - 1 - k : k;
      if (!end && (l.dtype[i] != dt || l.numel[i] == 0 || lies_apart(l, i))) continue;
      if (t.count == kClipTensors || (end && t.count > 0)) {
        if (backwards) {
          std::reverse(t.src, t.src + t.count);
          std::reverse(t.dst, t.dst + t.count);
          std::reverse(t.numel, t.numel + t.count);
        }
        int64_t chunks = 0, elems = 0;
        for (int j = 0; j < t.count; ++j) {
          chunks += (t.numel[j] + chunk - 1) / chunk;
          elems += t.numel[j];
          t.chunk_end[j] = chunks;
        }
        // the list's last kKeepBytes, to a chunk
        const int64_t cut = bytes - kKeepBytes - before;
        t.keep = cut <= 0 ? 0 : std::min(chunks, cut / (chunk * es));
        before += elems * es;
        const hipError_t e = fn(t, dt);
        if (e != hipSuccess) return e;
        t.count = 0;
      }
      if (end) break;
      t.src[t.count] = l.src ? l.src[i] : nullptr;
      t.dst[t.count] = l.dst ? l.dst[i] : nullptr;
      t.numel[t.count] = l.numel[i];
      ++t.count;
    }
  }
  return hipSuccess;
}

// The same for the tables of matrices whose rows lie apart.
template <typename F>
hipError_t for_row_tables(const ClipList& l, int num_cus, F fn) {
  if (!l.cols) return hipSuccess;
  int64_t total = 0;
  for (int64_t i = 0; i < l.count; ++i)
    if (lies_apart(l, i)) total += l.numel[i];
  for (int dt : {DT_F32, DT_F16, DT_BF16}) {
    ClipRows t{};
    // a wave's piece: a quarter of a workgroup's chunk
    t.chunk = chunk_elems(total, dtype_bytes(dt), num_cus) / (THREADS / 64);
    for (int64_t i = 0; i <= l.count; ++i) {
      const bool end = i == l.count;
      if (!end && (l.dtype[i] != dt || l.numel[i] == 0 || !lies_apart(l, i))) continue;
      if (t.count == kClipMatrices || (end && t.count > 0)) {
        const hipError_t e = fn(t, dt);
        if (e != hipSuccess) return e;
        t.count = 0;
      }
      if (end) break;
      const int k = t.count++;
      t.src[k] = l.src ? l.src[i] : nullptr;
      t.dst[k] = l.dst ? l.dst[i] : nullptr;
      t.cols[k] = l.cols[i];
      t.rows[k] = l.numel[i] / l.cols[i];
      t.ld[k] = l.ld ? l.ld[i] : 0;
      t.ld_out[k] = l.ld_out ? l.ld_out[i] : 0;
      const int64_t parts = (t.cols[k] + t.chunk - 1) / t.chunk, per = t.chunk / t.cols[k];
      t.chunk_end[k] = (k ? t.chunk_end[k - 1] : 0) + (parts > 1 ? t.rows[k] * parts : (t.rows[k] + per - 1) / per);
    }
  }
  return hipSuccess;
}

int grid_of(const ClipTable& t, int num_cus) {
  return (int)std::min<int64_t>(t.chunk_end[t.count - 1], (int64_t)num_cus * 8);
}
int grid_of(const ClipRows& t, int num_cus) {
  const int64_t waves = THREADS / 64;
  return (int)std::min<int64_t>((t.chunk_end[t.count - 1] + waves - 1) / waves, (int64_t)num_cus * 8);
}

template <bool INF>
hipError_t grad_norm_t(const ClipList& l, double max_norm, float* norm, double* partial, hipStream_t stream,
                       int num_cus) {
  int n = 0;
  hipError_t e = for_tables(l, num_cus, false, [&](const ClipTable& t, int dt) {
    const int g = grid_of(t, num_cus);
    double* out = partial + n;
    n += g;
    if (dt == DT_F32)
      hipLaunchKernelGGL((norm_kernel<float, INF>), dim3(g), dim3(THREADS), 0, stream, t, out);
    else if (dt == DT_F16)
      hipLaunchKernelGGL((norm_kernel<_Float16, INF>), dim3(g), dim3(THREADS), 0, stream, t, out);
    else
      hipLaunchKernelGGL((norm_kernel<__bf16, INF>), dim3(g), dim3(THREADS), 0, stream, t, out);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  e = for_row_tables(l, num_cus, [&](const ClipRows& t, int dt) {
    const int g = grid_of(t, num_cus);
    double* out = partial + n;
    n += g;
    if (dt == DT_F32)
      hipLaunchKernelGGL((norm_rows_kernel<float, INF>), dim3(g), dim3(THREADS), 0, stream, t, out);
    else if (dt == DT_F16)
      hipLaunchKernelGGL((norm_rows_kernel<_Float16, INF>), dim3(g), dim3(THREADS), 0, stream, t, out);
    else
      hipLaunchKernelGGL((norm_rows_kernel<__bf16, INF>), dim3(g), dim3(THREADS), 0, stream, t, out);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  if (!l.dst || n == 0) {
    hipLaunchKernelGGL((norm_only_kernel<INF>), dim3(1), dim3(THREADS), 0, stream, partial, n, norm);
    return hipGetLastError();
  }
  int64_t bytes = 0;
  for (int64_t i = 0; i < l.count; ++i) bytes += l.numel[i] * dtype_bytes(l.dtype[i]);
  const bool past = bytes > kPastBytes;
  bool first = true;
  e = for_row_tables(l, num_cus, [&](const ClipRows& t, int dt) {
    const int g = grid_of(t, num_cus);
    float* out = first ? norm : nullptr;
    first = false;
    if (dt == DT_F32)
      hipLaunchKernelGGL((scale_rows_kernel<float, INF>), dim3(g), dim3(THREADS), 0, stream, t, partial, n, max_norm, out);
    else if (dt == DT_F16)
      hipLaunchKernelGGL((scale_rows_kernel<_Float16, INF>), dim3(g), dim3(THREADS), 0, stream, t, partial, n, max_norm,
                         out);
    else
      hipLaunchKernelGGL((scale_rows_kernel<__bf16, INF>), dim3(g), dim3(THREADS), 0, stream, t, partial, n, max_norm,
                         out);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  return for_tables(l, num_cus, true, [&](const ClipTable& t, int dt) {
    const int g = grid_of(t, num_cus);
    float* out = first ? norm : nullptr;
    first = false;
    if (dt == DT_F32)
      hipLaunchKernelGGL((scale_kernel<float, INF>), dim3(g), dim3(THREADS), 0, stream, t, partial, n, max_norm, past,
                         out);
    else if (dt == DT_F16)
      hipLaunchKernelGGL((scale_kernel<_Float16, INF>), dim3(g), dim3(THREADS), 0, stream, t, partial, n, max_norm,
                         past, out);
    else
      hipLaunchKernelGGL((scale_kernel<__bf16, INF>), dim3(g), dim3(THREADS), 0, stream, t, partial, n, max_norm, past,
                         out);
    return hipGetLastError();
  });
}

}  // namespace

size_t grad_norm_workspace(const ClipList& l, int num_cus) {
  size_t n = 0;
  (void)for_tables(l, num_cus, false, [&](const ClipTable& t, int) {
    n += (size_t)grid_of(t, num_cus);
    return hipSuccess;
  });
  (void)for_row_tables(l, num_cus, [&](const ClipRows& t, int) {
    n += (size_t)grid_of(t, num_cus);
    return hipSuccess;
  });
  return n * sizeof(double);
}

hipError_t launch_grad_norm(const ClipList& l, bool inf, double max_norm, float* norm, void* workspace,
                            hipStream_t stream, int num_cus) {
  return inf ? grad_norm_t<true>(l, max_norm, norm, (double*)workspace, stream, num_cus)
             : grad_norm_t<false>(l, max_norm, norm, (double*)workspace, stream, num_cus);
}

}  // namespace coalesce
