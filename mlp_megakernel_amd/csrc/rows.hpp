// Rows of a matrix as the row-wise kernels read and write them: 8 consecutive
// columns per access, through a buffer resource that ends with the row, so a
// lane past the row's end needs no branch: it reads zeros and writes nothing.
#pragma once
#include "common.hpp"

namespace coalesce {
namespace {

// 8 values as they lie in memory.
template <typename T>
struct Raw8 {
  u32x4 q[sizeof(T) / 2];
};

template <typename T>
struct Row {
  __amdgpu_buffer_rsrc_t r;
  int cols;

  // The resource ends at a multiple of 4 bytes: loads are checked by whole
  // 4-byte words, so an odd number of 16-bit columns lets the last word in whole
  // (load() clears its upper half), and stores leave that word out (store()
  // writes its lower half by itself).
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t make(const void* base, int64_t ld, int64_t row, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)((const T*)base + row * ld), 0, bytes, 0x00020000);
  }
  static __device__ __forceinline__ Row in(const void* base, int64_t ld, int64_t row, int cols) {
    return Row{make(base, ld, row, ((uint32_t)cols * (uint32_t)sizeof(T) + 3u) & ~3u), cols};
  }
  static __device__ __forceinline__ Row out(void* base, int64_t ld, int64_t row, int cols) {
    return Row{make(base, ld, row, (uint32_t)cols * (uint32_t)sizeof(T) & ~3u), cols};
  }

  __device__ __forceinline__ Raw8<T> load(int n) const {
    Raw8<T> x;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      x.q[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, n * (int)sizeof(T) + 16 * i, 0, 0));
    return x;
  }
  // The values of load(n) in a row of so many columns.
  static __device__ __forceinline__ void widen(Raw8<T> x, int n, int cols, float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
      if (cols & 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + 2 * j + 1 == cols) x.q[0][j] &= 0xffffu;
      }
      typedef T t8 __attribute__((ext_vector_type(8)));
      const t8 t = __builtin_bit_cast(t8, x.q[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (float)t[e];
    } else {
      // (whole vectors: __builtin_bit_cast of an element reads the first one)
      const f32x4 lo = __builtin_bit_cast(f32x4, x.q[0]), hi = __builtin_bit_cast(f32x4, x.q[1]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = lo[e], v[4 + e] = hi[e];
    }
  }
  __device__ __forceinline__ void read(int n, float (&v)[8]) const { widen(load(n), n, cols, v); }

  // One rounding, to nearest even.  `base` is the row's first element (for the
  // odd last column).
  __device__ __forceinline__ void store(int n, const float (&v)[8], T* base) const {
    if constexpr (sizeof(T) == 2) {
      typedef T t8 __attribute__((ext_vector_type(8)));
      t8 t;
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = (T)v[e];
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, t), r, n * 2, 0, 0);
      if (cols & 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + 2 * j + 1 == cols) base[n + 2 * j] = t[2 * j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        __builtin_amdgcn_raw_buffer_store_b128(
            __builtin_bit_cast(u32x4, (f32x4){v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]}), r, n * 4 + 16 * i, 0, 0);
    }
  }
};

// A launch's arguments in the kernel-argument segment, behind an opaque copy of the
// pointer: each place loads what it needs (a scalar load that the cache serves)
// instead of all of it living in scalar registers, whose spills a loop would read
// back by vector instructions.
template <typename P>
using ArgsOf = const __attribute__((address_space(4))) P*;
template <typename P>
__device__ __forceinline__ ArgsOf<P> again(ArgsOf<P> k) {
  asm volatile("" : "+s"(k));
  return k;
}

// A vector of N values of a type that the launch names (a uniform branch).
template <typename T>
__device__ __forceinline__ void read_vec(const void* v, bool f32, int n, int N, float (&w)[8]) {
  if (f32)
    Row<float>::in(v, 0, 0, N).read(n, w);
  else
    Row<T>::in(v, 0, 0, N).read(n, w);
}

// Launches count the threads of a dimension in 32 bits, so many blocks go over two.
inline dim3 blocks_grid(int64_t blocks) {
  const int64_t x = blocks < (int64_t(1) << 21) ? blocks : int64_t(1) << 21;
  return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}
__device__ __forceinline__ int64_t block_no() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// The sum over a wave, in a fixed order, by the data-parallel row shifts and
// broadcasts (six additions, no LDS); every lane gets it.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp0(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp0<0x111, 0xf>(v);  // from 1, 2, 4 and 8 lanes below in the row of 16
  v += dpp0<0x112, 0xf>(v);
  v += dpp0<0x114, 0xf>(v);
  v += dpp0<0x118, 0xf>(v);
  v += dpp0<0x142, 0xa>(v);  // lane 15 of a row to the next, rows 1 and 3
  v += dpp0<0x143, 0xc>(v);  // lane 31 to rows 2 and 3
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

}  // namespace
}  // namespace coalesce
