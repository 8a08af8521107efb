// Forward of the feed-forward operators for few rows (up to 64 tokens): what
// costs there is reading the weights once, and the launches.
//
// A workgroup owns a strip of SN output columns (of both matrices of a gated
// product) and deals the K steps to its waves in turn, so every strip is one
// workgroup's, the workgroups sweep the weights in order, and one launch does it
// all, the epilogue included.  A wave
// streams its part of the weights through a private ring of D stages in LDS
// (32 k x SN columns each, 16-byte direct copies) and never meets a barrier
// until the end: it waits for its own oldest stage by the count of copies in
// flight, takes the fragments with transposing reads, and refills the slot.  X
// goes the same way, 16 rows x 32 k per copy, laid out as the MFMA operand.
// Rows past M and k past K read as zero by the buffers' ranges, except k past
// K inside a row of X, which the last step masks.  At the end the waves' fp32
// accumulators meet in LDS and are added in wave order.
#pragma once
#include "gemm16_core.hpp"

namespace coalesce {
namespace {

// NB matrices, MT 16-row blocks, SN columns, NW waves, D stages.
template <int NB_, int MT_, int SN_, int NW_, int D_>
struct FewGeo {
  static constexpr int NB = NB_, MT = MT_, SN = SN_, NW = NW_, D = D_;
  static constexpr int FK = 32;
  static constexpr int NT = SN / 16;
  static constexpr int CPR = SN / 8;                 // 16-byte chunks per weight row
  static constexpr int CB = FK * SN * 2 / 1024;      // 1 KB copies per matrix and stage
  static constexpr int C = NB * CB + MT;             // copies per stage
  static constexpr int STAGE = C * 1024;             // bytes
  static constexpr int RING = D * STAGE;
  // accumulators meet in LDS MR row blocks at a time
  static constexpr int BLOCK = NB * NT * 1024;       // bytes of one wave's accumulators per row block
  static constexpr int MR = MT * NW * BLOCK <= 131072 ? MT : MT / 2;
  static constexpr int LDS = NW * RING > MR * NW * BLOCK ? NW * RING : MR * NW * BLOCK;
  static_assert(MR * NW * BLOCK <= 131072 && LDS <= 160 * 1024 && (D - 1) * C < 64, "few-row plan");
};

// Chunk c of weight row k sits at slot c ^ few_swz(k).
template <int CPR>
__device__ __forceinline__ int few_swz(int k) {
  if constexpr (CPR == 8)
    return swzB<8>(k);
  else if constexpr (CPR == 4)  // 64-byte rows
    return ((k >> 3) & 1) << 1;
  else
    return 0;
}

template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <typename T, typename TO, int EPI, typename G>
__global__ __launch_bounds__(G::NW * 64) void few_kernel(TileOp p) {
  __shared__ __attribute__((aligned(1024))) char few_lds[G::LDS];
  constexpr int NB = G::NB, MT = G::MT, NT = G::NT, NW = G::NW, D = G::D, FK = G::FK;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // The hardware hands workgroups to the 8 XCDs in turn; each XCD takes a run
  // of neighbouring strips, so strips that share 128-byte lines share an L2.
  const int per_xcd = (int)(gridDim.x >> 3);
  const int strip = (int)(blockIdx.x & 7) * per_xcd + (int)(blockIdx.x >> 3);
  if (strip * (int64_t)G::SN >= p.N) return;
  const int n0 = strip * G::SN;
  const int steps = (p.K + FK - 1) / FK;
  char* const ring = few_lds + w * G::RING;
  const uint32_t ring_at = lds_addr(ring);

  // lane offsets of a copy: weights, CPR chunks per row; X, row lane & 15
  const uint32_t ldb_b = (uint32_t)p.ldb * 2u, lda_b = (uint32_t)p.lda * 2u;
  constexpr int RPC = 64 / G::CPR;  // weight rows per copy
  uint32_t boff[G::CB];
#pragma unroll
  for (int j = 0; j < G::CB; ++j) {
    const int k = j * RPC + lane / G::CPR;
    boff[j] = (uint32_t)k * ldb_b + (uint32_t)(((lane % G::CPR) ^ few_swz<G::CPR>(k)) * 16);
  }
  const uint32_t aoff = (uint32_t)(lane & 15) * lda_b + (uint32_t)((lane >> 4) * 16);
  const int cols = min(G::SN, p.N - n0);
  const uint32_t row_bytes = (uint32_t)((cols + 7) & ~7) * 2u;

  auto rsrc = [](const char* q, uint32_t bytes) {
    const uint64_t v = (uint64_t)(uintptr_t)q;
    return (u32x4){(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v),
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) & 0xffffu,
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
  };
  // K step s into ring slot `slot`; a step past the last reads nothing
  // (ranges of 0), which keeps the count of copies per step the same.
  auto issue = [&](int s, int slot) {
    const int k0 = s * FK;
    const int rows = s < steps ? min(FK, p.K - k0) : 0;
    const uint32_t nb = rows > 0 ? (uint32_t)(rows - 1) * ldb_b + row_bytes : 0u;
    uint32_t at = ring_at + (uint32_t)(slot * G::STAGE);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const u32x4 r = rsrc((const char*)((const T*)p.b[i] + (int64_t)k0 * p.ldb + n0), nb);
#pragma unroll
      for (int j = 0; j < G::CB; ++j) {
        dma16_buf(r, boff[j], 0u, at);
        at += 1024u;
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int left = min(16, p.M - 16 * i);  // rows of this block
      const uint32_t na = rows > 0 && left > 0 ? (uint32_t)(left - 1) * lda_b + (uint32_t)((rows + 7) & ~7) * 2u : 0u;
      const u32x4 r = rsrc((const char*)((const T*)p.a[0] + (int64_t)(16 * i) * p.lda + k0), na);
      dma16_buf(r, aoff, 0u, at);
      at += 1024u;
    }
  };

  f32x4 acc[NB][NT][MT];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[i][t][m] = (f32x4){0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int d = 0; d < D; ++d) issue(w + d * NW, d);
  int slot = 0;
  for (int s = w; s < steps; s += NW) {
    wait_copies<(D - 1) * G::C>();
    const char* st = ring + slot * G::STAGE;
    const int q = lane & 15, g = lane >> 4;
    i16x8 fx[MT], fb[NB][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m) fx[m] = *(const i16x8*)(st + NB * G::CB * 1024 + m * 1024 + lane * 16);
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        i16x4 h[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int k = 8 * g + 4 * u + (q >> 2);
          const int x = 16 * t + 4 * (q & 3);
          h[u] = lds_read_tr16(st + i * G::CB * 1024 + k * (G::SN * 2) + (((x >> 3) ^ few_swz<G::CPR>(k)) << 4) +
                               ((x & 7) << 1));
        }
        fb[i][t] = (i16x8){h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
      }
    // k past K inside a row of X may hold anything
    const int kl = p.K - s * FK - 8 * g;  // valid k of this lane's eight
    if (p.K - s * FK < FK) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e >= kl) fx[m][e] = 0;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot is read: refill it
    issue(s + D * NW, slot);
    slot = slot + 1 == D ? 0 : slot + 1;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[i][t][m] = mfma16x16x32(fb[i][t], fx[m], acc[i][t][m], T());
  }
  wait_copies<0>();  // no copy may land after the LDS changes hands

  const int q = lane & 15, g = lane >> 4;
#pragma unroll
  for (int r0 = 0; r0 < MT; r0 += G::MR) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < G::MR; ++m)
          *(f32x4*)(few_lds + (((w * G::MR + m) * NT + t) * NB + i) * 1024 + lane * 16) = acc[i][t][r0 + m];
    __syncthreads();
    // unit of the rest: one 16 x 16 block of the output
    for (int u = w; u < G::MR * NT; u += NW) {
      const int m = u / NT, t = u % NT;
      const int row = 16 * (r0 + m) + q, n = n0 + 16 * t + 4 * g;
      f32x4 z[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        z[i] = *(const f32x4*)(few_lds + ((m * NT + t) * NB + i) * 1024 + lane * 16);
#pragma unroll
        for (int v = 1; v < NW; ++v)
          z[i] += *(const f32x4*)(few_lds + (((v * G::MR + m) * NT + t) * NB + i) * 1024 + lane * 16);
      }
      if (row >= p.M || n >= p.N) continue;
      const int valid = min(4, p.N - n);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        if (p.bias[i]) z[i] += load4<T>((const T*)p.bias[i] + n, valid);
        if (p.Z[i]) store4<T>((T*)p.Z[i] + (int64_t)row * p.ldz + n, z[i], valid);
      }
      f32x4 o = (f32x4){0.f, 0.f, 0.f, 0.f};
      if (EPI == EPI_RESID && p.R) o = load4<TO>((const TO*)p.R + (int64_t)row * p.ldr + n, valid);
      const f32x4 f = act_any(p.act, z[0]);
      o = EPI == EPI_GATED ? f * z[NB - 1] : o + f;
      store4<TO>((TO*)p.Y[0] + (int64_t)row * p.ldy + n, o, valid);
    }
  }
}

template <typename T, typename TO, int EPI, typename G>
hipError_t few_launch(const TileOp& o, hipStream_t stream) {
  const unsigned strips = (unsigned)(((o.N + G::SN - 1) / G::SN + 7) / 8 * 8);  // whole rounds of the 8 XCDs
  hipLaunchKernelGGL((few_kernel<T, TO, EPI, G>), dim3(strips), dim3(G::NW * 64), 0, stream, o);
  return hipGetLastError();
}

// The ring is as deep as 160 KB allow: a compute unit needs some 60 KB in
// flight to draw its share of the memory's rate.
template <typename T, typename TO, int EPI, int SN>
hipError_t few_rows(const TileOp& o, hipStream_t stream) {
  constexpr int NB = EPI == EPI_GATED ? 2 : 1, KB = NB * SN / 16;  // KB: 1 KB copies of weights per stage
  if (o.M <= 16) return few_launch<T, TO, EPI, FewGeo<NB, 1, SN, 8, 20 / (KB + 1)>>(o, stream);
  if (o.M <= 32) return few_launch<T, TO, EPI, FewGeo<NB, 2, SN, 8, 20 / (KB + 2)>>(o, stream);
  if constexpr (KB == 8)
    return few_launch<T, TO, EPI, FewGeo<NB, 4, SN, 4, 3>>(o, stream);
  else
    return few_launch<T, TO, EPI, FewGeo<NB, 4, SN, 8, 20 / (KB + 4)>>(o, stream);
}

template <typename T, typename TO, int EPI>
hipError_t launch_few(const TileOp& o, int strip, hipStream_t stream) {
  if (strip == 64) return few_rows<T, TO, EPI, 64>(o, stream);
  if (strip == 32) return few_rows<T, TO, EPI, 32>(o, stream);
  return few_rows<T, TO, EPI, 16>(o, stream);
}

}  // namespace
}  // namespace coalesce
