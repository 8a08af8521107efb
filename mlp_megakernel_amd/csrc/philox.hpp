// The counter-based generator of the dropout mask: Philox4x32-10 (Salmon,
// Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", SC 2011).
// Element (m, n) of a matrix takes word n % 4 of the block whose counter is
// (n / 4, m, offset low, offset high) and whose key is the seed, so its fate
// depends on nothing but its place: not on the pitch, the type, the launch or
// the rows beside it, and the backward finds the forward's mask without storing
// it.
#pragma once
#include "block.hpp"
#include "common.hpp"

namespace coalesce {
namespace {

// Ten rounds; a round's two 32 x 32 -> 64-bit products are one instruction each.
// 8192 x 4096 bf16, operands that change from call to call: with a residual 36.5 us without
// rounds, 37.0 with 7 and 37.2 with 10; without one 24.4, 25.0 and 28.0.
__device__ __forceinline__ u32x4 philox(u32x4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * c[0], b = (uint64_t)0xCD9E8D57u * c[2];
    c = (u32x4){(uint32_t)(b >> 32) ^ c[1] ^ k0, (uint32_t)b, (uint32_t)(a >> 32) ^ c[3] ^ k1, (uint32_t)a};
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// What a launch needs of its mask, in scalar registers.
struct DropKey {
  uint32_t k0, k1, o0, o1, last;
  float scale;
};
template <typename D>  // Drop, in either address space
__device__ __forceinline__ DropKey drop_key(const D& d) {
  uint64_t seed = d.seed, offset = d.offset;
  if (d.device_seed) {
    seed = d.device_seed[0];
    offset = d.device_seed[1];
  }
  return DropKey{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)offset, (uint32_t)(offset >> 32), d.last, d.scale};
}

// Columns n .. n + 7 of row m (n a multiple of 8): kept values times the scale,
// 0 for the others, whatever they were (also NaN and infinities).
__device__ __forceinline__ void drop8(const DropKey& d, uint32_t m, uint32_t n, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const u32x4 w = philox((u32x4){(n >> 2) + h, m, d.o0, d.o1}, d.k0, d.k1);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * h + e] = w[e] > d.last ? v[4 * h + e] * d.scale : 0.0f;
  }
}

}  // namespace
}  // namespace coalesce
