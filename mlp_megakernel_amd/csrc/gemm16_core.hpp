// The 16-bit MFMA tile machinery of the feed-forward operators: one workgroup
// tile kernel over operands in either orientation, with the epilogue as a
// template argument (ffn_gemm.hip, ffn_bwd.hip), and the building blocks it
// shares with the plain fused GEMM (gemm16.hip).
//
//   acc[m][n] = sum_k Am[m][k] Bn[k][n]
//
// Am is the m side, Bn the n side.  Each side's tile is kept in LDS the way it
// lies in memory (Lay):
//   LAY_K  the contraction index is contiguous (X in X W, W in dZ W^T): rows of
//          64 k, fragments are 128-bit LDS reads;
//   LAY_X  the free index is contiguous (W in X W, both sides of X^T dZ): 64
//          rows of the tile's width, fragments come from the transposing LDS
//          read.
// So all three products of a layer (X W, dZ W^T, X^T dZ) run from the caller's
// row-major matrices without a transposed copy.  The schedule is the one of the
// plain fused GEMM: two LDS stages of a 64-deep K step, filled by direct
// 16-byte copies two steps ahead; each 32-deep slice issued as groups of
// {copies, MFMAs, a share of the next slice's fragment reads}; persistent
// workgroups whose next tile's copies start while the last stores drain.
#pragma once
#include <atomic>

#include "common.hpp"
#include "launch.hpp"

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

// Uniform (SGPR) 64-bit base for a direct copy.
__device__ __forceinline__ const void* uniform_ptr(const void* p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (const void*)(uintptr_t)(((uint64_t)hi << 32) | lo);
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16-byte direct copy: global (SGPR base + per-lane 32-bit offset) -> LDS
// (wave-uniform byte address + 16 * lane).
__device__ __forceinline__ void dma16_off(const void* base, uint32_t off, uint32_t lds) {
  // one wait state between the M0 write and the LDS-DMA instruction that reads it
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}

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

// 4 consecutive elements as fp32 (0 past `valid`); src is 4-element aligned.
template <typename T>
__device__ __forceinline__ f32x4 load4(const T* src, int valid) {
  f32x4 v = (f32x4){0.f, 0.f, 0.f, 0.f};
  if (valid >= 4) {
    typedef T t4 __attribute__((ext_vector_type(4)));
    const t4 x = *(const t4*)src;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = (float)x[r];
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < valid) v[r] = (float)src[r];
  }
  return v;
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


enum Lay { LAY_K = 0, LAY_X = 1 };
enum Epi { EPI_STORE = 0, EPI_RESID = 1, EPI_GATED = 2 };

// Tile geometry: BM x BN accumulators per workgroup, NW waves in a WGM x
// NW / WGM grid.  NSUB = 2: the n side's tile is two sub-tiles of BN / 2
// columns, the same columns of two matrices (the gated product: a wave holds
// both products of its WN / 2 columns, so act(g) * u needs no exchange).
// MINW is the launch-bounds floor of waves per SIMD.
template <int BM_, int BN_, int NW_, int WGM_, int MINW_, int NSUB_>
struct TileGeo {
  static constexpr int BM = BM_, BN = BN_, NW = NW_, WGM = WGM_, MINW = MINW_, NSUB = NSUB_;
  static constexpr int THREADS = NW * 64;
  static constexpr int WGN = NW / WGM;
  static constexpr int WM = BM / WGM, WN = BN / WGN;  // wave tile (WN over all sub-tiles)
  static constexpr int MT = WM / 16, NT = WN / 16;    // 16-wide sub-blocks per wave
  static constexpr int SUBN = BN / NSUB;              // columns of one n-side sub-tile
  static constexpr int ON = SUBN;                     // output columns per workgroup tile
  static constexpr int WNO = WN / NSUB, NTO = NT / NSUB;
  static constexpr int CA = BM / 8 / NW;              // 1 KB copies per wave and K step
  static constexpr int CBS = SUBN / 8 / NW;
  static constexpr int CB = CBS * NSUB, C = CA + CB;
  static constexpr int NG = MT < NT ? MT : NT;        // MFMA groups per slice
  static constexpr int NI = MT < NT ? NT : MT;        // MFMAs per group
  static constexpr bool OUTER_N = NT <= MT;           // groups run over the n side's fragments
  static constexpr int STAGE_A = BM * BK, STAGE_B = BN * BK;
  static constexpr int LDS_ELEMS = 2 * (STAGE_A + STAGE_B);
  static_assert(CA * NW * 8 == BM && CBS * NW * 8 == SUBN && CA > 0 && CBS > 0, "copy plan does not cover the tile");
  static_assert((NG == 4 && (NI == 8 || NI == 4)) || (NG == 2 && (NI == 2 || NI == 4)), "no read plan for this wave tile");
};

// One side of the product as the copies see it: `p` is the matrix, x0 the
// tile's first free index, X the free extent, K the contraction extent.
struct Side {
  const void* p;
  int64_t ld;
  int x0, X;
};

// 1 KB copy j of wave w of a BX-wide tile: (LDS element offset, per-lane byte
// offset from the tile's base at k0).  32-bit arithmetic is exact: the host
// checks that 256 rows fit in 32 bits.
template <typename T, Lay L, int BX>
__device__ __forceinline__ uint32_t copy_offset(const Side& s, int g, int lane) {
  const uint32_t ld_b = (uint32_t)s.ld * (uint32_t)sizeof(T);
  if constexpr (L == LAY_K) {
    const int row = g * 8 + (lane >> 3);
    const int c = (lane & 7) ^ swzA(row);
    const int gx = min(s.x0 + row, s.X - 1);
    return (uint32_t)(gx - s.x0) * ld_b + (uint32_t)(c * 8 * (int)sizeof(T));
  } else {
    constexpr int CPR = BX / 8, RPC = 64 / CPR;
    const int row = g * RPC + lane / CPR;
    const int c = (lane & (CPR - 1)) ^ swzB<CPR>(row);
    const int gx = min(s.x0 + c * 8, ((s.X - 1) >> 3) << 3);
    return (uint32_t)row * ld_b + (uint32_t)((gx - s.x0) * (int)sizeof(T));
  }
}

template <typename T, Lay L>
__device__ __forceinline__ const void* side_base(const Side& s, int k0) {
  if constexpr (L == LAY_K)
    return uniform_ptr((const T*)s.p + (int64_t)s.x0 * s.ld + k0);
  else
    return uniform_ptr((const T*)s.p + (int64_t)k0 * s.ld + s.x0);
}

// Masked register loads of the same 16 bytes (elements at k >= K become 0):
// the last, partial K step.
template <typename T, Lay L, int BX>
__device__ __forceinline__ i16x8 tail_chunk(const Side& s, int g, int lane, int k0, int K) {
  i16x8 v = (i16x8){0, 0, 0, 0, 0, 0, 0, 0};
  if constexpr (L == LAY_K) {
    const int row = g * 8 + (lane >> 3);
    const int k = k0 + ((lane & 7) ^ swzA(row)) * 8;
    const int gx = min(s.x0 + row, s.X - 1);
    if (k < K) {
      v = *(const i16x8*)((const T*)s.p + (int64_t)gx * s.ld + k);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e >= K) v[e] = 0;
    }
  } else {
    constexpr int CPR = BX / 8, RPC = 64 / CPR;
    const int row = g * RPC + lane / CPR;
    const int c = (lane & (CPR - 1)) ^ swzB<CPR>(row);
    const int gx = min(s.x0 + c * 8, ((s.X - 1) >> 3) << 3);
    if (k0 + row < K) v = *(const i16x8*)((const T*)s.p + (int64_t)(k0 + row) * s.ld + gx);
  }
  return v;
}

// MFMA operand fragment: free index x0 + (lane & 15), k = 32 ks + 8 (lane >> 4) + e.
template <typename T, Lay L, int BX>
__device__ __forceinline__ i16x8 read_frag(const T* t, int ks, int x0, int lane) {
  if constexpr (L == LAY_K) {
    const int x = x0 + (lane & 15);
    const int c = (4 * ks + (lane >> 4)) ^ swzA(x);
    return *(const i16x8*)(t + x * BK + c * 8);
  } else {
    constexpr int CPR = BX / 8;
    const int q = lane & 15;
    const int x = x0 + 4 * (q & 3);
    i16x4 h[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = 32 * ks + 8 * (lane >> 4) + 4 * i + (q >> 2);
      h[i] = lds_read_tr16(t + k * BX + (((x >> 3) ^ swzB<CPR>(k)) << 3) + (x & 7));
    }
    return (i16x8){h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
  }
}

// Everything a tile's K loop needs besides the accumulators.
struct TileAt {
  int m0, n0;   // first row and output column
  int pair;     // product of a batch of two
  int s0, ns;   // first K step (over all segments) and number of steps
  int split;
};

template <typename G>
struct TileFrags {
  i16x8 n[G::NT];
  i16x8 m[G::MT];
};

template <typename T, typename TO, Lay LA, Lay LB, int EPI, typename G>
struct Tile {
  // ---- K steps ---------------------------------------------------------
  static __device__ __forceinline__ int steps_per_seg(const TileOp& p) { return (p.K + BK - 1) / BK; }
  static __device__ __forceinline__ void step_at(const TileOp& p, int s, int& seg, int& k0) {
    const int kt = steps_per_seg(p);
    seg = s >= kt ? 1 : 0;
    k0 = (s - seg * kt) * BK;
  }
  static __device__ __forceinline__ Side side_a(const TileOp& p, const TileAt& at, int seg) {
    return Side{seg ? p.a[1] : p.a[0], seg ? p.lda[1] : p.lda[0], at.m0, p.M};
  }
  static __device__ __forceinline__ Side side_b(const TileOp& p, const TileAt& at, int seg, int sub) {
    const int i = seg | at.pair | sub;  // at most one of them is used by any launch
    return Side{i ? p.b[1] : p.b[0], i ? p.ldb[1] : p.ldb[0], at.n0, p.N};
  }

  // Copy j (0 .. C - 1) of K step s into stage (a, b).
  static __device__ __forceinline__ void copy(const TileOp& p, const TileAt& at, int j, int seg, int k0, T* a, T* b,
                                              int wu, int lane) {
    if (j < G::CA) {
      const Side s = side_a(p, at, seg);
      const int g = wu * G::CA + j;
      dma16_off(side_base<T, LA>(s, k0), copy_offset<T, LA, G::BM>(s, g, lane), lds_addr(a) + (uint32_t)g * 1024u);
    } else {
      const int jj = j - G::CA, sub = jj / G::CBS;
      const Side s = side_b(p, at, seg, sub);
      const int g = wu * G::CBS + jj % G::CBS;
      dma16_off(side_base<T, LB>(s, k0), copy_offset<T, LB, G::SUBN>(s, g, lane),
                lds_addr(b) + (uint32_t)(sub * G::SUBN * BK * (int)sizeof(T)) + (uint32_t)g * 1024u);
    }
  }

  static __device__ __forceinline__ void tail(const TileOp& p, const TileAt& at, int seg, int k0, T* a, T* b, int w,
                                              int lane) {
    i16x8 ra[G::CA], rb[G::CB];
    const Side sa = side_a(p, at, seg);
#pragma unroll
    for (int j = 0; j < G::CA; ++j) ra[j] = tail_chunk<T, LA, G::BM>(sa, w * G::CA + j, lane, k0, p.K);
#pragma unroll
    for (int j = 0; j < G::CB; ++j)
      rb[j] = tail_chunk<T, LB, G::SUBN>(side_b(p, at, seg, j / G::CBS), w * G::CBS + j % G::CBS, lane, k0, p.K);
#pragma unroll
    for (int j = 0; j < G::CA; ++j) *(i16x8*)(a + (w * G::CA + j) * 512 + lane * 8) = ra[j];
#pragma unroll
    for (int j = 0; j < G::CB; ++j)
      *(i16x8*)(b + (j / G::CBS) * G::SUBN * BK + (w * G::CBS + j % G::CBS) * 512 + lane * 8) = rb[j];
  }

  // K step s, all copies at once (a tile's first two steps).
  static __device__ __forceinline__ void fill(const TileOp& p, const TileAt& at, int s, T* a, T* b, int wu, int lane) {
    int seg, k0;
    step_at(p, s, seg, k0);
    if (k0 + BK <= p.K) {
#pragma unroll
      for (int j = 0; j < G::C; ++j) copy(p, at, j, seg, k0, a, b, wu, lane);
    } else {
      tail(p, at, seg, k0, a, b, wu, lane);
    }
  }

  // ---- fragments and MFMAs ---------------------------------------------
  static __device__ __forceinline__ i16x8 frag_m(const T* a, int ks, int wm, int i, int lane) {
    return read_frag<T, LA, G::BM>(a, ks, wm * G::WM + 16 * i, lane);
  }
  static __device__ __forceinline__ i16x8 frag_n(const T* b, int ks, int wn, int i, int lane) {
    const int sub = i / G::NTO;
    return read_frag<T, LB, G::SUBN>(b + sub * G::SUBN * BK, ks, wn * G::WNO + 16 * (i % G::NTO), lane);
  }

  // One 32-deep slice: NG groups of {a share of the copies of K step k + 2,
  // NI MFMAs, a share of the next slice's fragment reads, those its first
  // group needs first}, a scheduling fence after each.  On the last step the
  // "next" reads fetch stale but in-bounds LDS and are unused.
  static __device__ __forceinline__ void slice(const TileFrags<G>& cur, f32x4 (&acc)[G::NT][G::MT], TileFrags<G>& nxt,
                                               const T* ra, const T* rb, int rks, int wm, int wn, int lane, bool cp,
                                               const TileOp& p, const TileAt& at, int seg, int k0, T* ca, T* cb,
                                               int wu) {
    auto read_outer = [&](int i) {
      if constexpr (G::OUTER_N)
        nxt.n[i] = frag_n(rb, rks, wn, i, lane);
      else
        nxt.m[i] = frag_m(ra, rks, wm, i, lane);
    };
    auto read_inner = [&](int i) {
      if constexpr (G::OUTER_N)
        nxt.m[i] = frag_m(ra, rks, wm, i, lane);
      else
        nxt.n[i] = frag_n(rb, rks, wn, i, lane);
    };
#pragma unroll
    for (int g = 0; g < G::NG; ++g) {
      if (cp) {
#pragma unroll
        for (int j = G::C * g / G::NG; j < G::C * (g + 1) / G::NG; ++j) copy(p, at, j, seg, k0, ca, cb, wu, lane);
      }
#pragma unroll
      for (int i = 0; i < G::NI; ++i) {
        const int t = G::OUTER_N ? g : i, s = G::OUTER_N ? i : g;
        acc[t][s] = mfma16x16x32(cur.n[t], cur.m[s], acc[t][s], T());
      }
      // the reads after the MFMAs: a fragment of the next slice may then take
      // the registers of one the MFMAs above were the last use of
      __builtin_amdgcn_sched_barrier(0);
      if (g == 0) {
        read_outer(0);
#pragma unroll
        for (int i = 0; i < (G::NI < 4 ? G::NI : 4); ++i) read_inner(i);
      } else if (G::NI == 8) {
        if (g == 1) {
#pragma unroll
          for (int i = 4; i < 8; ++i) read_inner(i);
        } else if (g == 2) {
          read_outer(1);
          read_outer(2);
        } else {
          read_outer(3);
        }
      } else {
        read_outer(g);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // ---- epilogue ----------------------------------------------------------
  // Rows [wr0, wr0 + WM) x columns [wc0, wc0 + WNO) of one output matrix from
  // value(t, s, m, n, valid), the 4 consecutive columns n.. of row m.  A
  // 16-bit block that lies whole inside the matrix is staged in the wave's
  // own LDS region and stored as full row segments; others are stored from
  // the registers.
  template <typename TS, typename F>
  static __device__ __forceinline__ void put(TS* Y, int64_t ldy, const TileOp& p, int wr0, int wc0, bool inside,
                                             char* region, int lane, F value) {
    const int q = lane & 15, b = lane >> 4;
    if constexpr (sizeof(TS) == 2) {
      if (inside) {
        constexpr int ROWB = G::WNO * 2, CPR = ROWB / 16, RPI = 64 / CPR;
        typedef TS to4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int t = 0; t < G::NTO; ++t) {
          const int chunk = 2 * t + (b >> 1);
#pragma unroll
          for (int s = 0; s < G::MT; ++s) {
            const int row = 16 * s + q;
            const f32x4 v = value(t, s, wr0 + row, wc0 + 16 * t + 4 * b, 4);
            const to4 o = (to4){(TS)v[0], (TS)v[1], (TS)v[2], (TS)v[3]};
            *(to4*)(region + row * ROWB + ((chunk ^ stage_swz<ROWB>(row)) << 4) + ((b & 1) << 3)) = o;
          }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        const int rsub = lane / CPR, c = lane % CPR;
#pragma unroll
        for (int i = 0; i < G::WM / RPI; ++i) {
          const int row = RPI * i + rsub;
          const u32x4 v = *(const u32x4*)(region + row * ROWB + ((c ^ stage_swz<ROWB>(row)) << 4));
          *(u32x4*)(Y + (int64_t)(wr0 + row) * ldy + wc0 + 8 * c) = v;
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        return;
      }
    }
#pragma unroll
    for (int t = 0; t < G::NTO; ++t) {
      const int n = wc0 + 16 * t + 4 * b;
      if (n >= p.N) continue;
      const int valid = min(4, p.N - n);
#pragma unroll
      for (int s = 0; s < G::MT; ++s) {
        const int m = wr0 + 16 * s + q;
        if (m < p.M) store4<TS>(Y + (int64_t)m * ldy + n, value(t, s, m, n, valid), valid);
      }
    }
  }

  template <int ACT>
  static __device__ __forceinline__ void finish(const TileOp& p, const TileAt& at, f32x4 (&acc)[G::NT][G::MT], int wr0,
                                                int wc0, bool inside, char* region, int lane) {
    constexpr bool O16 = sizeof(TO) == 2;
    // + bias, in place
#pragma unroll
    for (int t = 0; t < G::NT; ++t) {
      const T* bias = (const T*)(t / G::NTO ? p.bias[1] : p.bias[0]);
      if (bias) {
        const int n = wc0 + 16 * (t % G::NTO) + 4 * (lane >> 4);
        const f32x4 bv = load4<T>(bias + (n < p.N ? n : 0), min(4, p.N - n));
#pragma unroll
        for (int s = 0; s < G::MT; ++s) acc[t][s] += bv;
      }
    }
    // the stored pre-activations of a training forward, one rounding each
    if (p.Z[0]) {
      put<T>((T*)p.Z[0], p.ldz, p, wr0, wc0, inside, region, lane,
             [&](int t, int s, int, int, int) { return acc[t][s]; });
      if constexpr (EPI == EPI_GATED)
        put<T>((T*)p.Z[1], p.ldz, p, wr0, wc0, inside, region, lane,
               [&](int t, int s, int, int, int) { return acc[t + G::NTO][s]; });
    }
    if constexpr (EPI == EPI_GATED) {
      put<TO>((TO*)p.Y[0], p.ldy[0], p, wr0, wc0, inside, region, lane, [&](int t, int s, int, int, int) {
        f32x4 o;
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = apply_act<ACT, O16>(acc[t][s][r]) * acc[t + G::NTO][s][r];
        return o;
      });
    } else {
      const TO* R = (const TO*)p.R;
      put<TO>((TO*)p.Y[0], p.ldy[0], p, wr0, wc0, inside, region, lane, [&](int t, int s, int m, int n, int valid) {
        f32x4 o = (f32x4){0.f, 0.f, 0.f, 0.f};
        if (R) o = load4<TO>(R + (int64_t)m * p.ldr + n, valid);
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] += apply_act<ACT, O16>(acc[t][s][r]);
        return o;
      });
    }
  }

  static __device__ __forceinline__ void epilogue(const TileOp& p, const TileAt& at, f32x4 (&acc)[G::NT][G::MT], int wm,
                                                  int wn, int wu, int lane, char* lds) {
    const int wr0 = at.m0 + wm * G::WM, wc0 = at.n0 + wn * G::WNO;
    const bool inside = wr0 + G::WM <= p.M && wc0 + G::WNO <= p.N;
    char* region = lds + wu * (G::WM * G::WNO * 2);
    static_assert(G::NW * G::WM * G::WNO * 2 <= G::LDS_ELEMS * 2, "staging regions exceed the stages");
    if constexpr (EPI == EPI_STORE) {
#pragma unroll
      for (int sub = 0; sub < G::NSUB; ++sub) {
        const int i = at.pair | sub;
        TO* Y = (TO*)(i ? p.Y[1] : p.Y[0]) + (int64_t)at.split * p.split_stride;
        put<TO>(Y, i ? p.ldy[1] : p.ldy[0], p, wr0, wc0, inside, region, lane,
                [&](int t, int s, int, int, int) { return acc[t + sub * G::NTO][s]; });
      }
    } else {
      switch (p.act) {
        case ACT_GELU: finish<ACT_GELU>(p, at, acc, wr0, wc0, inside, region, lane); break;
        case ACT_SOFTPLUS: finish<ACT_SOFTPLUS>(p, at, acc, wr0, wc0, inside, region, lane); break;
        case ACT_RELU: finish<ACT_RELU>(p, at, acc, wr0, wc0, inside, region, lane); break;
        case ACT_SILU: finish<ACT_SILU>(p, at, acc, wr0, wc0, inside, region, lane); break;
        default: finish<ACT_NONE>(p, at, acc, wr0, wc0, inside, region, lane); break;
      }
    }
  }

  // Unit of work v: one tile of one range of K steps.  The two products of a
  // batch lie side by side in the tile order, so they share the m side.
  static __device__ __forceinline__ TileAt locate(const TileOp& p, int64_t v) {
    TileAt at;
    const int tn_all = p.tiles_n * p.batch;
    const int64_t tiles = (int64_t)p.tiles_m * tn_all;
    at.split = (int)(v / tiles);
    int tm, tn;
    tile_coords((int)(v - at.split * tiles), p.tiles_m, tn_all, p.group_m, tm, tn);
    at.pair = tn >= p.tiles_n ? 1 : 0;
    at.m0 = tm * G::BM;
    at.n0 = (tn - at.pair * p.tiles_n) * G::ON;
    const int64_t total = (int64_t)steps_per_seg(p) * p.segs;
    at.s0 = (int)(total * at.split / p.splits);
    at.ns = (int)(total * (at.split + 1) / p.splits) - at.s0;
    return at;
  }

  static __device__ __forceinline__ void run(const TileOp& p, T* lds) {
    T* const a0 = lds;
    T* const a1 = lds + G::STAGE_A;
    T* const b0 = lds + 2 * G::STAGE_A;
    T* const b1 = b0 + G::STAGE_B;
    const int64_t total = (int64_t)p.tiles_m * p.tiles_n * p.batch * p.splits;
    int64_t v = blockIdx.x;
    if (v >= total) return;
    const int lane0 = threadIdx.x & 63;
    const int wu = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wu % G::WGM, wn = wu / G::WGM;

    TileAt at = locate(p, v);
    if (at.ns > 0) fill(p, at, at.s0, a0, b0, wu, lane0);
    if (at.ns > 1) fill(p, at, at.s0 + 1, a1, b1, wu, lane0);
    while (true) {
      // the lane index through an opaque copy: everything derived from it is
      // recomputed per tile instead of being held across the K loop
      int lane = lane0;
      asm volatile("" : "+v"(lane));
      f32x4 acc[G::NT][G::MT];
#pragma unroll
      for (int t = 0; t < G::NT; ++t)
#pragma unroll
        for (int s = 0; s < G::MT; ++s) acc[t][s] = (f32x4){0.f, 0.f, 0.f, 0.f};
      TileFrags<G> f0, f1;
      if (at.ns > 0) {
        wait_vmcnt0();
        __syncthreads();
#pragma unroll
        for (int i = 0; i < G::NT; ++i) f0.n[i] = frag_n(b0, 0, wn, i, lane);
#pragma unroll
        for (int i = 0; i < G::MT; ++i) f0.m[i] = frag_m(a0, 0, wm, i, lane);
      }
      // Per K step k (stage cur; the other stage holds step k + 1 or is
      // filling): slice 0 on f0 while f1 is read; barrier (cur is free, step
      // k + 1 has landed); slice 1 on f1 while step k + 2 is copied into cur
      // and f0 of step k + 1 is read.
      for (int kt = 0; kt < at.ns; kt += 2) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int k = kt + half;
          if (k < at.ns) {
            T* const ca = half ? a1 : a0;
            T* const cb = half ? b1 : b0;
            T* const na = half ? a0 : a1;
            T* const nb = half ? b0 : b1;
            slice(f0, acc, f1, ca, cb, 1, wm, wn, lane, false, p, at, 0, 0, ca, cb, wu);
            if (k + 1 < at.ns) {
              wait_vmcnt0();
              __syncthreads();
            }
            int seg = 0, k0 = 0;
            bool cp = false;
            if (k + 2 < at.ns) {
              step_at(p, at.s0 + k + 2, seg, k0);
              cp = k0 + BK <= p.K;
              if (!cp) tail(p, at, seg, k0, ca, cb, wu, lane);
            }
            slice(f1, acc, f0, na, nb, 0, wm, wn, lane, cp, p, at, seg, k0, ca, cb, wu);
          }
        }
      }
      __syncthreads();  // every wave is past its last fragment read
      epilogue(p, at, acc, wm, wn, wu, lane, (char*)lds);
      lds_barrier();  // the LDS is free; the stores may still be in flight
      v += gridDim.x;
      if (v >= total) break;
      at = locate(p, v);
      if (at.ns > 0) fill(p, at, at.s0, a0, b0, wu, lane);
      if (at.ns > 1) fill(p, at, at.s0 + 1, a1, b1, wu, lane);
    }
  }
};

template <typename T, typename TO, Lay LA, Lay LB, int EPI, typename G>
__global__ __launch_bounds__(G::THREADS, G::MINW) void tile_kernel(TileOp p) {
  __shared__ __attribute__((aligned(1024))) T lds[G::LDS_ELEMS];
  Tile<T, TO, LA, LB, EPI, G>::run(p, lds);
}

// Grid: min(#units of work, #CUs x workgroups per CU), the per-CU count from
// the runtime for the compiled kernel, cached per instantiation (atomic:
// concurrent first calls store the same value).
template <typename T, typename TO, Lay LA, Lay LB, int EPI, typename G>
hipError_t launch_tile(TileOp p, hipStream_t stream, int num_cus) {
  p.tiles_m = (p.M + G::BM - 1) / G::BM;
  p.tiles_n = (p.N + G::ON - 1) / G::ON;
  if (p.group_m <= 0) p.group_m = 8;
  static std::atomic<int> per_cu_cache{0};
  int per_cu = per_cu_cache.load(std::memory_order_relaxed);
  if (per_cu == 0) {
    int n = 0;
    hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, tile_kernel<T, TO, LA, LB, EPI, G>, G::THREADS, 0);
    if (e != hipSuccess) return e;
    per_cu = n > 0 ? n : 1;
    per_cu_cache.store(per_cu, std::memory_order_relaxed);
  }
  const int64_t total = (int64_t)p.tiles_m * p.tiles_n * p.batch * p.splits;
  const int64_t cap = (int64_t)num_cus * per_cu;
  hipLaunchKernelGGL((tile_kernel<T, TO, LA, LB, EPI, G>), dim3((unsigned)(total < cap ? total : cap)),
                     dim3(G::THREADS), 0, stream, p);
  return hipGetLastError();
}

}  // namespace
}  // namespace coalesce
