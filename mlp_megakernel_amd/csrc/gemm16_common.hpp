// What the two 16-bit MFMA GEMM kernels share (gemm16.hip, gemm16_core.hpp): the
// LDS swizzles, the barrier of the pipeline, the stores of an epilogue.
#pragma once
#include "common.hpp"

namespace coalesce {
namespace {

constexpr int BK = 64;

// LDS swizzles, in 16-byte chunks.  LAY_K rows (64 k, 128 B = 8 chunks): chunk
// c of row m sits at slot c ^ swzA(m): a 128-bit read by 16 lanes (rows
// m0..m0+15, one chunk) hits 16 distinct 16-byte slots of a 256-byte window,
// and any 8 consecutive rows hit 8 distinct slots of a 128-byte window.
// LAY_X rows (CPR chunks of the free index): chunk c of row k sits at slot c ^
// swzB<CPR>(k): a transposing read by 32 lanes (rows k0..k0+3 and
// k0+8..k0+11, two chunks, two 8-byte halves) hits 32 distinct 8-byte slots of
// a 256-byte window (which holds two rows when they are 128 bytes long).
// Neither depends on the sub-tile index, the slice or the half of a
// transposing read, so those stay immediate offsets of the LDS reads.
__device__ __forceinline__ int swzA(int m) { return ((m >> 1) & 7) ^ ((m & 1) << 2); }
template <int CPR>
__device__ __forceinline__ int swzB(int k) {
  if constexpr (CPR >= 16)
    return ((k & 3) << 1) | (((k >> 3) & 1) << 3);
  else  // 128-byte rows: a 256-byte window holds two rows, k and k ^ 1
    return (((k >> 1) & 1) << 1) | (((k >> 3) & 1) << 2);
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// Workgroup barrier for LDS reuse: the wave's own LDS accesses are complete
// (lgkmcnt 0) but its global stores and direct copies may still be in
// flight (no vmcnt wait, unlike __syncthreads' fence); the "memory" clobber
// keeps the compiler from moving memory accesses across it.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
#pragma clang diagnostic pop

template <typename TO>
__device__ __forceinline__ void store4(TO* dst, f32x4 v, int valid) {
  if constexpr (sizeof(TO) == 2) {
    typedef TO to4 __attribute__((ext_vector_type(4)));
    const to4 o = (to4){(TO)v[0], (TO)v[1], (TO)v[2], (TO)v[3]};
    if (valid >= 4) {
      *(to4*)dst = o;
    } else {
      for (int r = 0; r < valid; ++r) dst[r] = o[r];
    }
  } else {
    if (valid >= 4) {
      *(f32x4*)dst = v;
    } else {
      for (int r = 0; r < valid; ++r) dst[r] = v[r];
    }
  }
}

// Swizzle of an epilogue staging row of ROWB bytes (64, 128 or 256), in
// 16-byte chunks: both the 8-byte writes of 16 rows and the 16-byte
// row-contiguous reads spread over the banks.
template <int ROWB>
__device__ __forceinline__ int stage_swz(int row) {
  if constexpr (ROWB == 64)
    return (row >> 2) & 3;
  else if constexpr (ROWB == 128)
    return (row >> 1) & 7;
  else
    return row & 15;
}

}  // namespace
}  // namespace coalesce
