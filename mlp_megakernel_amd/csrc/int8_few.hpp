// The 8-bit products for few rows (up to 64 tokens): what costs there is reading
// the weights once.
//
// The weights lie channel by channel (N x K), so a fragment of the matrix
// instruction is 16 consecutive bytes of a row; but its lanes go over the rows
// first, and loads into registers in that order look up one cache line per lane: 16
// bytes a cycle and compute unit, weights and tokens together (64 x 4096 x 16384, weights
// that the caches may hold: 40 us).  So both go through LDS by direct copies of whole
// 128-byte lines (20 us; weights that change from call to call 21 to 23, 1 x 16384 x 4096
// gated 27, 5.0 TB/s, and 1 x 2731 x 1001 3.8).
// A workgroup owns 16 NT channels (of both matrices of a gated product) and deals
// the K steps of 128 to its waves in turn; a wave streams its steps through a private
// ring of D stages and never meets a barrier until the end: it waits for its own
// oldest stage by the count of copies in flight, takes the fragments and refills the
// slot.  At the end the waves' int32 sums meet in LDS; they do not depend on their
// order, so a row's result is the one that any other kernel gives.
// Rows past M and channels past N read as zero by the buffers' ranges; k past K
// inside a row of X is masked, which settles it for the weights too.
#pragma once
#include "gemm16_core.hpp"

namespace coalesce {
namespace {

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// dma16_buf for bytes that no other workgroup reads: the caches need not keep them.
__device__ __forceinline__ void dma16_once(u32x4 rsrc, uint32_t off, uint32_t shift, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %3 offen nt lds" ::"v"(off), "s"(rsrc),
               "s"(lds), "s"(shift)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// NB matrices, NT blocks of 16 channels of each, MH times 8 rows (1, 2, 4 or 8), NW
// waves, D stages.
template <int NB_, int NT_, int MH_, int NW_, int D_>
struct Few8Geo {
  static constexpr int NB = NB_, NT = NT_, MH = MH_, MT = (MH + 1) / 2, NW = NW_, D = D_, KB = NB * NT;
  static constexpr int C = 2 * KB + MH;  // 1 KB copies per stage: 8 rows of 128 bytes each
  static constexpr int STAGE = C * 1024, RING = D * STAGE;
  static constexpr int SUMS = NW * KB * MT * 1024;
  static constexpr int LDS = NW * RING > SUMS ? NW * RING : SUMS;
  static_assert(LDS <= 160 * 1024 && (D - 1) * C < 64, "few-row plan");
};

template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// ONCE: the weights go past the caches.
template <typename TO, int EPI, typename G, bool ONCE>
__global__ __launch_bounds__(G::NW * 64) void few8_kernel(TileOp p) {
  constexpr int NB = G::NB, NT = G::NT, MT = G::MT, NW = G::NW, D = G::D, KB = G::KB;
  __shared__ __attribute__((aligned(1024))) char few_lds[G::LDS];
  const int lane = threadIdx.x & 63, q = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (int)blockIdx.x * 16 * NT;
  const int steps = (p.K + 127) / 128;
  const uint32_t row_bytes = (uint32_t)((p.K + 15) & ~15);
  const uint32_t lda = (uint32_t)p.lda * 2u, ldb = (uint32_t)p.ldb * 2u;  // pitches count pairs
  char* const ring = few_lds + w * G::RING;
  const uint32_t ring_at = lds_addr(ring);

  // 16 rows of a matrix from row r0 on, as far as it has them.
  auto rows16 = [&](const void* base, uint32_t ld, int64_t r0, int all) {
    const int left = (int)min((int64_t)16, (int64_t)all - r0);
    const uint64_t v = (uint64_t)(uintptr_t)((const char*)base + (left > 0 ? r0 : 0) * (int64_t)ld);
    return (u32x4){(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v),
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) & 0xffffu,
                   left > 0 ? (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(left - 1) * ld + row_bytes)) : 0u,
                   0x00020000u};
  };
  u32x4 rb[KB], rx[MT];
#pragma unroll
  for (int i = 0; i < KB; ++i) rb[i] = rows16(p.b[i / NT], ldb, n0 + 16 * (i % NT), p.N);
#pragma unroll
  for (int m = 0; m < MT; ++m) rx[m] = rows16(p.a[0], lda, 16 * m, p.M);
  // lane offsets of the two copies of 16 rows: eight lanes per row, the 16-byte pieces
  // in the tiles' order (swzA)
  uint32_t ob[2], ox[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = 8 * h + (lane >> 3);
    const uint32_t at = (uint32_t)((lane & 7) ^ swzA(row)) * 16u;
    ob[h] = (uint32_t)row * ldb + at;
    ox[h] = (uint32_t)row * lda + at;
  }
  // K step s into ring slot `slot`; a step past the last lies outside every range and
  // reads nothing, which keeps the count of copies per step the same.
  auto issue = [&](int s, int slot) {
    const uint32_t shift = s < steps ? (uint32_t)s * 128u : 1u << 30;
    uint32_t at = ring_at + (uint32_t)(slot * G::STAGE);
#pragma unroll
    for (int i = 0; i < KB; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (ONCE)
          dma16_once(rb[i], ob[h], shift, at);
        else
          dma16_buf(rb[i], ob[h], shift, at);
        at += 1024u;
      }
#pragma unroll
    for (int h = 0; h < G::MH; ++h) {
      dma16_buf(rx[h / 2], ox[h % 2], shift, at);
      at += 1024u;
    }
  };

  i32x4 acc[KB][MT];
#pragma unroll
  for (int i = 0; i < KB; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = (i32x4){0, 0, 0, 0};
#pragma unroll
  for (int d = 0; d < D; ++d) issue(w + d * NW, d);
  int slot = 0;
  for (int s = w; s < steps; s += NW) {
    wait_copies<(D - 1) * G::C>();
    const char* st = ring + slot * G::STAGE;
    const int xr = G::MH == 1 ? q & 7 : q;  // (up to 8 rows: the other 8 results are no one's)
    i32x4 fb[KB][2], fx[MT][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int cb = q * 128 + ((4 * j + g) ^ swzA(q)) * 16, cx = xr * 128 + ((4 * j + g) ^ swzA(xr)) * 16;
#pragma unroll
      for (int i = 0; i < KB; ++i) fb[i][j] = *(const i32x4*)(st + i * 2048 + cb);
#pragma unroll
      for (int m = 0; m < MT; ++m) fx[m][j] = *(const i32x4*)(st + (KB + m) * 2048 + cx);
    }
    if ((s + 1) * 128 > p.K) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int left = p.K - s * 128 - 64 * j - 16 * g;  // valid bytes of this lane's sixteen
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int n = left - 4 * d;
          const int mask = n >= 4 ? -1 : n <= 0 ? 0 : (int)((1u << (8 * n)) - 1u);
#pragma unroll
          for (int m = 0; m < MT; ++m) fx[m][j][d] &= mask;
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot is read: refill it
    issue(s + D * NW, slot);
    slot = slot + 1 == D ? 0 : slot + 1;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < KB; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[i][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[i][j], fx[m][j], acc[i][m], 0, 0, 0);
  }
  wait_copies<0>();  // no copy may land after the LDS changes hands
  __syncthreads();
  i32x4(*const sums)[MT][KB][64] = (i32x4(*)[MT][KB][64])few_lds;
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

template <typename TO, int EPI, typename G, bool ONCE = false>
hipError_t few8_launch(const TileOp& o, hipStream_t stream) {
  hipLaunchKernelGGL((few8_kernel<TO, EPI, G, ONCE>), dim3((unsigned)((o.N + 16 * G::NT - 1) / (16 * G::NT))),
                     dim3(G::NW * 64), 0, stream, o);
  return hipGetLastError();
}

// The choice is plan_int8's.
template <typename TO, int EPI>
hipError_t launch_few8(const TileOp& o, Few8Kind kind, hipStream_t stream) {
  constexpr int NB = EPI == EPI_INT8_GATED ? 2 : 1;
  switch (kind) {
    case FEW8_8_WIDE:
      if constexpr (NB == 1) return few8_launch<TO, EPI, Few8Geo<NB, 1, 1, 8, 3>>(o, stream);
      break;
    case FEW8_8_LONG:
      if constexpr (NB == 2) return few8_launch<TO, EPI, Few8Geo<NB, 1, 1, 8, 2>, true>(o, stream);
      break;
    case FEW8_8_ONCE: return few8_launch<TO, EPI, Few8Geo<NB, 1, 1, 4, 3>, true>(o, stream);
    case FEW8_8: return few8_launch<TO, EPI, Few8Geo<NB, 1, 1, 4, 3>>(o, stream);
    case FEW8_16_ONCE: return few8_launch<TO, EPI, Few8Geo<NB, 1, 2, 4, 2>, true>(o, stream);
    case FEW8_16: return few8_launch<TO, EPI, Few8Geo<NB, 1, 2, 4, 2>>(o, stream);
    case FEW8_32: return few8_launch<TO, EPI, Few8Geo<NB, 1, 4, 4, 2>>(o, stream);
    case FEW8_64: return few8_launch<TO, EPI, Few8Geo<NB, 1, 8, 4, 2>>(o, stream);
    case FEW8_64_PAIRS: return few8_launch<TO, EPI, Few8Geo<NB, 2, 8, 2 * NB, NB == 2 ? 2 : 3>>(o, stream);
    default: break;
  }
  return hipErrorInvalidValue;
}

}  // namespace
}  // namespace coalesce
