// The 16-bit MFMA tile machinery of the feed-forward operators: one workgroup
// tile kernel over operands in either orientation, with the epilogue as a
// template argument (ffn_forward.hpp, ffn_backward.hpp).
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
// plain fused GEMM: two (or three) LDS stages of a 64-deep K step, filled by direct
// 16-byte copies that many steps ahead; each 32-deep slice issued as groups of
// {copies, MFMAs, a share of the next slice's fragment reads}; persistent
// workgroups whose next tile's copies start while the last stores drain.
#pragma once
#include <atomic>

#include "ffn_act.hpp"
#include "gemm16_common.hpp"
#include "launch.hpp"

namespace coalesce {
namespace {

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16-byte direct copy through a buffer resource, at the lane's offset plus a
// uniform one, to LDS (wave-uniform byte address + 16 * lane): bytes at or past
// the resource's size read as zero, so a tile that overhangs its matrix needs no
// clamps.
__device__ __forceinline__ void dma16_buf(u32x4 rsrc, uint32_t off, uint32_t shift, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds" ::"v"(off), "s"(rsrc),
               "s"(lds), "s"(shift)
               : "memory", "m0");
}
#pragma clang diagnostic pop

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

enum Lay { LAY_K = 0, LAY_X = 1 };
enum Epi { EPI_STORE = 0, EPI_RESID = 1, EPI_GATED = 2 };

// Tile geometry: BM x BN accumulators per workgroup, NW waves in a WGM x
// NW / WGM grid, NS stages in LDS.  With two stages a copy has one K step's time
// to arrive, which a 256 x 256 tile covers; narrower tiles whose step is shorter
// than a trip to memory take three.  NSUB = 2: the n side's tile is two sub-tiles of BN / 2
// columns, the same columns of two matrices (the gated product: a wave holds
// both products of its WN / 2 columns, so act(g) * u needs no exchange).
// MINW is the launch-bounds floor of waves per SIMD.
template <int BM_, int BN_, int NW_, int WGM_, int MINW_, int NSUB_, int NS_ = 2>
struct TileGeo {
  static constexpr int BM = BM_, BN = BN_, NW = NW_, WGM = WGM_, MINW = MINW_, NSUB = NSUB_, NS = NS_;
  static constexpr int THREADS = NW * 64;
  static constexpr int WGN = NW / WGM;
  static constexpr int WM = BM / WGM, WN = BN / WGN;  // wave tile (WN over all sub-tiles)
  static constexpr int MT = WM / 16, NT = WN / 16;    // 16-wide sub-blocks per wave
  static constexpr int SUBN = BN / NSUB;              // columns of one n-side sub-tile
  static constexpr int ON = SUBN;                     // output columns per workgroup tile
  static constexpr int WNO = WN / NSUB, NTO = NT / NSUB;
  static constexpr int NCA = BM / 8;                  // 1 KB copies of the m side per K step,
  static constexpr int CA = (NCA + NW - 1) / NW;      // at most so many per wave
  static constexpr int CBS = SUBN / 8 / NW;
  static constexpr int CB = CBS * NSUB, C = CA + CB;
  static constexpr int NG = MT < NT ? MT : NT;        // MFMA groups per slice
  static constexpr int NI = MT < NT ? NT : MT;        // MFMAs per group
  static constexpr bool OUTER_N = NT <= MT;           // groups run over the n side's fragments
  // The last round of m-side copies may have more waves than rows are left:
  // their copies (out of the range, zeros) get room behind the tile's rows, or,
  // where three stages leave none, one place behind the stages.
  static constexpr bool ROOM = NS * (CA * NW * 8 + BN) * BK * 2 <= 160 * 1024;
  static constexpr int STAGE_A = (ROOM ? CA * NW * 8 : BM) * BK, STAGE_B = BN * BK;
  static constexpr int LDS_ELEMS = NS * (STAGE_A + STAGE_B);
  static_assert(NCA * 8 == BM && CBS * NW * 8 == SUBN, "copy plan does not cover the tile");
  static_assert(NS == 2 || NS == 3, "wait_steps keeps one later step in flight");
  static_assert(LDS_ELEMS * 2 + (ROOM ? 0 : 1024) <= 160 * 1024, "the stages exceed the LDS");
  static_assert(NG >= 2 && NI <= 8 && WM * WGM == BM && MT * 16 == WM && NT * 16 == WN,
                "no read plan for this wave tile");
};

// One side of the product as the copies see it: `p` is the matrix, x0 the
// tile's first free index, X the free extent, K the contraction extent.
struct Side {
  const void* p;
  int64_t ld;
  int x0, X;
};

// Rows of a tile in LDS that one 1 KB copy fills.
template <Lay L, int BX>
struct CopyRows {
  static constexpr int N = L == LAY_K ? 8 : 512 / BX;
};

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

// MFMA operand fragment i of a wave's N: free index x0 + 16 i + (lane & 15), k =
// 32 ks + 8 (lane >> 4) + e.  In LAY_X tiles the fragments of one row lie 32 i
// apart before the swizzle, which flips the same bits: their LDS addresses are
// one address with those bits flipped, formed per read where a wave holds
// eight (eight addresses would not fit in the registers beside the
// accumulators), and left to the compiler to keep where it holds fewer.
template <typename T, Lay L, int BX, int N>
__device__ __forceinline__ i16x8 read_frag(const T* t, int ks, int x0, int i, int lane) {
  if constexpr (L == LAY_K) {
    const int x = x0 + 16 * i + (lane & 15);
    const int c = (4 * ks + (lane >> 4)) ^ swzA(x);
    return *(const i16x8*)(t + x * BK + c * 8);
  } else {
    constexpr int CPR = BX / 8;
    const int q = lane & 15;
    const int k0 = 8 * (lane >> 4) + (q >> 2);
    i16x4 h[2];
    if constexpr (N == 8 && CPR >= 16) {
      // x0 is a multiple of 128, so i alone sets bits 1..3 of the chunk
      const int x = x0 + 4 * (q & 3);
      const uint32_t a0 =
          lds_addr(t) + (uint32_t)((k0 * BX + (((x >> 3) ^ swzB<CPR>(k0)) << 3) + (x & 7)) * (int)sizeof(T));
      uint32_t a;
      asm volatile("v_xor_b32 %0, %1, %2" : "=v"(a) : "i"(32 * i), "v"(a0));
#pragma unroll
      for (int u = 0; u < 2; ++u)
        h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) i16x4*)(uintptr_t)(a + (uint32_t)((32 * ks + 4 * u) * BX * (int)sizeof(T))));
    } else {
      const int x = x0 + 16 * i + 4 * (q & 3);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = 32 * ks + k0 + 4 * u;
        h[u] = lds_read_tr16(t + k * BX + (((x >> 3) ^ swzB<CPR>(k)) << 3) + (x & 7));
      }
    }
    return (i16x8){h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
  }
}

// The launch's arguments in the kernel-argument segment.  Code outside the K
// loop reads them through fresh(): an opaque copy of the pointer, so that each
// place loads what it needs instead of the whole struct living in scalar
// registers (where it would spill, and the spills' reloads would sit in the
// loop).
typedef const __attribute__((address_space(4))) TileOp* Args;
__device__ __forceinline__ Args fresh(Args k) {
  asm volatile("" : "+s"(k));
  return k;
}

// Where a tile lies and which K steps are its.
struct TileAt {
  int m0, n0;   // first row and output column
  int pair;     // product of a batch of two
  int split;
  int s0, s1;   // range of K steps over all segments
};
struct Range1 {
  int s, n;  // first K step and number of steps in one segment
};

template <typename G>
struct TileFrags {
  i16x8 n[G::NT];
  i16x8 m[G::MT];
};

// SEGS = 2: the K loop runs over two products, a[0] b[0] + a[1] b[1].
template <typename T, typename TO, Lay LA, Lay LB, int SEGS, int EPI, typename G>
struct Tile {
  static constexpr int RA = CopyRows<LA, G::BM>::N, RB = CopyRows<LB, G::SUBN>::N;
  static_assert(SEGS == 1 || G::NSUB == 1, "segments of a gated product are not implemented");

  // What the K loop needs of the tile, in scalar registers: the matrices at
  // the tile's first free index and k = 0, the bytes per k and per copy, and
  // the size of a full K step's part of the matrix (the buffer's range: rows
  // or columns outside the matrix lie past it or are never stored).
  struct Hot {
    const char* a;
    const char* b[G::NSUB];
    int64_t ka, kb;
    uint32_t ra, rb, na, nb;
    int K;
  };
  // Lane offset of a wave's copies, per side.
  struct Pats {
    uint32_t a, b;
  };
  // Sources of one K step.
  struct Step {
    u32x4 a, b[G::NSUB];
    int k0;
  };

  static __device__ __forceinline__ Side side_a(Args p, const TileAt& at, int seg) {
    return Side{p->a[SEGS == 2 ? seg : 0], p->lda, at.m0, p->M};
  }
  static __device__ __forceinline__ Side side_b(Args p, const TileAt& at, int seg, int sub) {
    return Side{p->b[SEGS == 2 ? seg : G::NSUB == 2 ? sub : at.pair], p->ldb, at.n0, p->N};
  }

  // Bytes from the first to behind the last one that a full K step reads.
  template <Lay L, int BX>
  static __device__ __forceinline__ uint32_t step_bytes(const Side& s) {
    const int x = min(BX, s.X - s.x0);
    if constexpr (L == LAY_K)
      return (uint32_t)((x - 1) * s.ld + BK) * (uint32_t)sizeof(T);
    else
      return (uint32_t)((BK - 1) * s.ld + ((x + 7) & ~7)) * (uint32_t)sizeof(T);
  }
  static __device__ __forceinline__ Hot hot(Args k, const TileAt& at, int seg) {
    const Args p = fresh(k);
    Hot h;
    h.K = p->K;
    h.ra = (uint32_t)(G::NW * RA * p->lda * (int)sizeof(T));
    h.rb = (uint32_t)(G::NW * RB * p->ldb * (int)sizeof(T));
    h.ka = (LA == LAY_K ? 1 : p->lda) * (int64_t)sizeof(T);
    h.kb = (LB == LAY_K ? 1 : p->ldb) * (int64_t)sizeof(T);
    const Side sa = side_a(p, at, seg);
    h.a = (const char*)((const T*)sa.p + (LA == LAY_K ? sa.x0 * sa.ld : (int64_t)sa.x0));
    h.na = step_bytes<LA, G::BM>(sa);
#pragma unroll
    for (int i = 0; i < G::NSUB; ++i) {
      const Side s = side_b(p, at, seg, i);
      h.b[i] = (const char*)((const T*)s.p + (LB == LAY_K ? s.x0 * s.ld : (int64_t)s.x0));
      h.nb = step_bytes<LB, G::SUBN>(s);
    }
    return h;
  }

  // ---- K steps ---------------------------------------------------------
  static __device__ __forceinline__ u32x4 rsrc(const char* p, uint32_t bytes) {
    const uint64_t v = (uint64_t)(uintptr_t)p;
    return (u32x4){(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v),
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) & 0xffffu,
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
  }
  static __device__ __forceinline__ Step step_at(const Hot& h, int s) {
    Step t;
    t.k0 = s * BK;
    t.a = rsrc(h.a + t.k0 * h.ka, h.na);
#pragma unroll
    for (int i = 0; i < G::NSUB; ++i) t.b[i] = rsrc(h.b[i] + t.k0 * h.kb, h.nb);
    return t;
  }

  // Copy j of wave wu fills rows from (j NW + wu) RPC on: the copies of a wave
  // differ by a whole number of NW RPC rows, a multiple of the swizzles'
  // period, so one lane offset per side serves them all and the rows are a
  // uniform offset.
  template <Lay L, int BX>
  static __device__ __forceinline__ uint32_t pattern(int64_t ld, int wu, int lane) {
    constexpr int RPC = CopyRows<L, BX>::N;
    static_assert(G::NW * RPC % 16 == 0, "the swizzles repeat every 16 rows");
    const uint32_t ld_b = (uint32_t)ld * (uint32_t)sizeof(T);
    if constexpr (L == LAY_K) {
      const int row = wu * RPC + (lane >> 3);
      return (uint32_t)row * ld_b + (uint32_t)((((lane & 7) ^ swzA(row)) * 8) * (int)sizeof(T));
    } else {
      constexpr int CPR = BX / 8;
      const int row = wu * RPC + lane / CPR;
      return (uint32_t)row * ld_b + (uint32_t)((((lane & (CPR - 1)) ^ swzB<CPR>(row)) * 8) * (int)sizeof(T));
    }
  }
  static __device__ __forceinline__ Pats patterns(Args k, int wu, int lane) {
    const Args p = fresh(k);
    return Pats{pattern<LA, G::BM>(p->lda, wu, lane), pattern<LB, G::SUBN>(p->ldb, wu, lane)};
  }

  // Copy j (0 .. C - 1) of a K step into stage (a, b).
  // The m side's stages lie first in the LDS, lds_stage is a's number.
  static __device__ __forceinline__ void copy(const Hot& h, const Pats& pt, const Step& st, int j, uint32_t lds_stage,
                                              T* a, T* b, int wu) {
    if (j < G::CA) {
      u32x4 r = st.a;
      uint32_t at = (uint32_t)(j * G::NW + wu) * 1024u;
      if (!G::ROOM && (j + 1) * G::NW > G::NCA) {
        // waves without a copy left copy zeros from an empty range, so that all
        // waves count the same number
        const bool mine = j * G::NW + wu < G::NCA;
        r[2] = mine ? r[2] : 0u;
        at = mine ? at : (uint32_t)(G::LDS_ELEMS * (int)sizeof(T)) - lds_stage * (uint32_t)(G::STAGE_A * (int)sizeof(T));
      }
      dma16_buf(r, pt.a, (uint32_t)j * h.ra, lds_addr(a) + at);
    } else {
      const int sub = (j - G::CA) / G::CBS, jj = (j - G::CA) % G::CBS;
      dma16_buf(st.b[sub], pt.b, (uint32_t)jj * h.rb,
                lds_addr(b) + (uint32_t)(sub * G::SUBN * BK * (int)sizeof(T)) + (uint32_t)(jj * G::NW + wu) * 1024u);
    }
  }
  // Waits until at most LATER later K steps' copies of this wave are in flight.
  template <int LATER>
  static __device__ __forceinline__ void wait_steps() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LATER * G::C) : "memory");
  }

  // The m side's copy j of wave w; past the last one it again (the same bytes
  // to the same place).  w comes in a vector register: a comparison with the
  // uniform wave number here makes the compiler keep the whole tile's addresses
  // in vector registers, read back to scalars at each copy.
  static __device__ __forceinline__ int m_chunk(int j, int w) {
    return G::ROOM || (j + 1) * G::NW <= G::NCA ? j * G::NW + w : min(j * G::NW + w, G::NCA - 1);
  }
  static __device__ __forceinline__ void tail(Args k, const TileAt& at, int seg, const Step& st, T* a, T* b, int w,
                                              int lane) {
    // the lane through an opaque copy: the addresses are formed here, not
    // carried in registers through the K loop
    asm volatile("" : "+v"(lane));
    int wv = w;
    asm volatile("" : "+v"(wv));
    const Args p = fresh(k);
    const int K = p->K;
    i16x8 ra[G::CA], rb[G::CB];
    const Side sa = side_a(p, at, seg);
#pragma unroll
    for (int j = 0; j < G::CA; ++j) ra[j] = tail_chunk<T, LA, G::BM>(sa, m_chunk(j, wv), lane, st.k0, K);
#pragma unroll
    for (int j = 0; j < G::CB; ++j)
      rb[j] = tail_chunk<T, LB, G::SUBN>(side_b(p, at, seg, j / G::CBS), j % G::CBS * G::NW + w, lane, st.k0, K);
#pragma unroll
    for (int j = 0; j < G::CA; ++j) *(i16x8*)(a + m_chunk(j, wv) * 512 + lane * 8) = ra[j];
#pragma unroll
    for (int j = 0; j < G::CB; ++j)
      *(i16x8*)(b + (j / G::CBS) * G::SUBN * BK + (j % G::CBS * G::NW + w) * 512 + lane * 8) = rb[j];
  }

  // K step s, all copies at once (a segment's first NS steps).
  static __device__ __forceinline__ void fill(Args k, const TileAt& at, int seg, const Hot& h, const Pats& pt, int s,
                                              uint32_t stage, T* a, T* b, int wu, int lane) {
    const Step st = step_at(h, s);
    if (st.k0 + BK <= h.K) {
#pragma unroll
      for (int j = 0; j < G::C; ++j) copy(h, pt, st, j, stage, a, b, wu);
    } else {
      tail(k, at, seg, st, a, b, wu, lane);
    }
  }

  // ---- fragments and MFMAs ---------------------------------------------
  static __device__ __forceinline__ i16x8 frag_m(const T* a, int ks, int wm, int i, int lane) {
    return read_frag<T, LA, G::BM, G::MT>(a, ks, wm * G::WM, i, lane);
  }
  static __device__ __forceinline__ i16x8 frag_n(const T* b, int ks, int wn, int i, int lane) {
    const int sub = i / G::NTO;
    return read_frag<T, LB, G::SUBN, G::NTO>(b + sub * G::SUBN * BK, ks, wn * G::WNO, i % G::NTO, lane);
  }

  // One 32-deep slice: NG groups of {a share of the copies of K step k + NS,
  // NI MFMAs, a share of the next slice's fragment reads, those its first
  // group needs first}, a scheduling fence after each.  On the last step the
  // "next" reads fetch stale but in-bounds LDS and are unused.
  static __device__ __forceinline__ void slice(const TileFrags<G>& cur, f32x4 (&acc)[G::NT][G::MT], TileFrags<G>& nxt,
                                               const T* ra, const T* rb, int rks, int wm, int wn, int lane, bool cp,
                                               const Hot& h, const Pats& pt, const Step& st, uint32_t stage, T* ca, T* cb,
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
        for (int j = G::C * g / G::NG; j < G::C * (g + 1) / G::NG; ++j) copy(h, pt, st, j, stage, ca, cb, wu);
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
      } else if (G::NI > 4) {
        // the rest of the inner side in group 1, the outer fragments spread
        // over the groups behind it
        if (g == 1) {
#pragma unroll
          for (int i = 4; i < G::NI; ++i) read_inner(i);
          if (G::NG == 2) read_outer(1);
        } else {
          constexpr int REST = G::NG - 1, LEFT = G::NG - 2;  // fragments, groups
#pragma unroll
          for (int i = 1 + ((g - 2) * REST + LEFT - 1) / (LEFT > 0 ? LEFT : 1);
               i < 1 + ((g - 1) * REST + LEFT - 1) / (LEFT > 0 ? LEFT : 1); ++i)
            read_outer(i);
        }
      } else {
        read_outer(g);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // ---- epilogue ----------------------------------------------------------
  // A wave's WM x WNO block of a 16-bit matrix into its staging region, whole
  // row segments at a time, in the places put() gives its own values.  (The
  // residual, read where it is added, came as 32-byte pieces of 16 rows per
  // load: 4096 x 4096 with K = 64 26.8 us, so 20.6, and 13 without a residual.)
  template <typename TS>
  static __device__ __forceinline__ void stage_rows(const TS* src, int64_t ld, char* region, int lane) {
    constexpr int ROWB = G::WNO * 2, CPR = ROWB / 16, RPI = 64 / CPR;
    const uint32_t ld_b = (uint32_t)ld * 2u;
    const u32x4 r = rsrc((const char*)src, (uint32_t)(G::WM - 1) * ld_b + (uint32_t)ROWB);
    const int rsub = lane / CPR, c = lane % CPR;
#pragma unroll
    for (int i = 0; i < G::WM / RPI; ++i)
      dma16_buf(r, (uint32_t)rsub * ld_b + (uint32_t)((c ^ stage_swz<ROWB>(RPI * i + rsub)) << 4),
                (uint32_t)(RPI * i) * ld_b, lds_addr(region) + (uint32_t)i * 1024u);
    wait_vmcnt0();
  }

  // Rows [wr0, wr0 + WM) x columns [wc0, wc0 + WNO) of one output matrix:
  // prep(t, n, valid) once per 16-wide sub-block gives what value(c, t, s, m,
  // n, valid, cell), the 4 consecutive columns n.. of row m, needs of its
  // columns; cell is their place in the staging region, if they go through it.
  // A 16-bit block that lies whole inside the matrix is staged in the wave's
  // own LDS region and stored as full row segments; others are stored from
  // the registers.
  template <typename TS, typename P, typename F>
  static __device__ __forceinline__ void put(TS* Y, int64_t ldy, Args p, int wr0, int wc0, bool inside,
                                             char* region, int lane, P prep, F value) {
    const int q = lane & 15, b = lane >> 4;
    if constexpr (sizeof(TS) == 2) {
      if (inside) {
        constexpr int ROWB = G::WNO * 2, CPR = ROWB / 16, RPI = 64 / CPR;
        typedef TS to4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int t = 0; t < G::NTO; ++t) {
          const int chunk = 2 * t + (b >> 1);
          const auto c = prep(t, wc0 + 16 * t + 4 * b, 4);
#pragma unroll
          for (int s = 0; s < G::MT; ++s) {
            const int row = 16 * s + q;
            char* cell = region + row * ROWB + ((chunk ^ stage_swz<ROWB>(row)) << 4) + ((b & 1) << 3);
            const f32x4 v = value(c, t, s, wr0 + row, wc0 + 16 * t + 4 * b, 4, cell);
            const to4 o = (to4){(TS)v[0], (TS)v[1], (TS)v[2], (TS)v[3]};
            *(to4*)cell = o;
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
      if (n >= p->N) continue;
      const int valid = min(4, p->N - n);
      const auto c = prep(t, n, valid);
#pragma unroll
      for (int s = 0; s < G::MT; ++s) {
        const int m = wr0 + 16 * s + q;
        if (m < p->M) store4<TS>(Y + (int64_t)m * ldy + n, value(c, t, s, m, n, valid, (const char*)nullptr), valid);
      }
    }
  }

  static __device__ __forceinline__ f32x4 bias4(const void* bias, int n, int valid) {
    return bias ? load4<T>((const T*)bias + n, valid) : (f32x4){0.f, 0.f, 0.f, 0.f};
  }

  static __device__ __forceinline__ void epilogue(Args k, const TileAt& at, f32x4 (&acc)[G::NT][G::MT], int wm,
                                                  int wn, int wu, int lane, char* lds) {
    const Args p = fresh(k);
    const int wr0 = at.m0 + wm * G::WM, wc0 = at.n0 + wn * G::WNO;
    const bool inside = wr0 + G::WM <= p->M && wc0 + G::WNO <= p->N;
    char* region = lds + wu * (G::WM * G::WNO * 2);
    static_assert(G::NW * G::WM * G::WNO * 2 <= G::LDS_ELEMS * 2, "staging regions exceed the stages");
    constexpr bool O16 = sizeof(TO) == 2;
    auto none = [](int, int, int) { return 0; };
    if constexpr (EPI == EPI_STORE) {
#pragma unroll
      for (int sub = 0; sub < G::NSUB; ++sub) {
        const int i = at.pair | sub;
        TO* Y = (TO*)(i ? p->Y[1] : p->Y[0]) + (int64_t)at.split * p->split_stride;
        put<TO>(Y, p->ldy, p, wr0, wc0, inside, region, lane, none,
                [&](int, int t, int s, int, int, int, const char*) { return acc[t + sub * G::NTO][s]; });
      }
    } else {
      const int act = p->act;
      auto bias_g = [&](int, int n, int valid) { return bias4(p->bias[0], n, valid); };
      auto bias_u = [&](int, int n, int valid) { return bias4(p->bias[1], n, valid); };
      // the stored pre-activations of a training forward, one rounding each
      if (p->Z[0]) {
        put<T>((T*)p->Z[0], p->ldz, p, wr0, wc0, inside, region, lane, bias_g,
               [&](f32x4 c, int t, int s, int, int, int, const char*) { return acc[t][s] + c; });
        if constexpr (EPI == EPI_GATED)
          put<T>((T*)p->Z[1], p->ldz, p, wr0, wc0, inside, region, lane, bias_u,
                 [&](f32x4 c, int t, int s, int, int, int, const char*) { return acc[t + G::NTO][s] + c; });
      }
      if constexpr (EPI == EPI_GATED) {
        struct Pair {
          f32x4 g, u;
        };
        put<TO>((TO*)p->Y[0], p->ldy, p, wr0, wc0, inside, region, lane,
                [&](int t, int n, int valid) { return Pair{bias_g(t, n, valid), bias_u(t, n, valid)}; },
                [&](Pair c, int t, int s, int, int, int, const char*) {
                  const f32x4 g = acc[t][s] + c.g, u = acc[t + G::NTO][s] + c.u;
                  return act_any(act, g) * u;
                });
      } else {
        const TO* R = (const TO*)p->R;
        if (O16 && R && inside) stage_rows<TO>(R + (int64_t)wr0 * p->ldr + wc0, p->ldr, region, lane);
        put<TO>((TO*)p->Y[0], p->ldy, p, wr0, wc0, inside, region, lane, bias_g,
                [&](f32x4 c, int t, int s, int m, int n, int valid, const char* cell) {
                  const f32x4 z = acc[t][s] + c;
                  f32x4 o = (f32x4){0.f, 0.f, 0.f, 0.f};
                  if (R) o = load4<TO>(cell ? (const TO*)cell : R + (int64_t)m * p->ldr + n, valid);
                  return o + act_any(act, z);
                });
      }
    }
  }

  // Unit of work v: one tile of one range of K steps.  The two products of a
  // batch lie side by side in the tile order, so they share the m side.
  static __device__ __forceinline__ TileAt locate(Args k, int64_t v) {
    const Args p = fresh(k);
    TileAt at;
    const int tn_all = p->tiles_n * p->batch;
    const int64_t tiles = (int64_t)p->tiles_m * tn_all;
    at.split = (int)(v / tiles);
    int tm, tn;
    tile_coords((int)(v - at.split * tiles), p->tiles_m, tn_all, p->group_m, tm, tn);
    at.pair = tn >= p->tiles_n ? 1 : 0;
    at.m0 = tm * G::BM;
    at.n0 = (tn - at.pair * p->tiles_n) * G::ON;
    const int64_t total = (int64_t)((p->K + BK - 1) / BK) * SEGS;
    at.s0 = (int)(total * at.split / p->splits);
    at.s1 = (int)(total * (at.split + 1) / p->splits);
    return at;
  }
  // The part of the tile's K steps that lies in a segment.
  static __device__ __forceinline__ Range1 part(const TileAt& at, const Hot& h, int seg) {
    if constexpr (SEGS == 1) return Range1{at.s0, at.s1 - at.s0};
    const int kt = (h.K + BK - 1) / BK;
    const int lo = max(at.s0 - seg * kt, 0), hi = min(at.s1 - seg * kt, kt);
    return Range1{lo, max(hi - lo, 0)};
  }

  static __device__ __forceinline__ void run(Args k, T* lds) {
    const Args p = fresh(k);
    auto sa = [&](int i) { return lds + i * G::STAGE_A; };
    auto sb = [&](int i) { return lds + G::NS * G::STAGE_A + i * G::STAGE_B; };
    auto fill_first = [&](const TileAt& at, int seg, const Hot& h, const Range1& r, const Pats& pt, int wu, int lane) {
#pragma unroll
      for (int i = 0; i < G::NS; ++i)
        if (i < r.n) fill(k, at, seg, h, pt, r.s + i, (uint32_t)i, sa(i), sb(i), wu, lane);
    };
    const int64_t total = (int64_t)p->tiles_m * p->tiles_n * p->batch * p->splits;
    int64_t v = blockIdx.x;
    if (v >= total) return;
    const int lane0 = threadIdx.x & 63;
    const int wu = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wu % G::WGM, wn = wu / G::WGM;

    TileAt at = locate(k, v);
    Hot h = hot(k, at, 0);
    Range1 r = part(at, h, 0);
    const Pats pt = patterns(k, wu, lane0);
    fill_first(at, 0, h, r, pt, wu, lane0);
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
      // One pass of the pipeline per segment (a second one refills the stages:
      // one exposed latency per tile, against pointers of both segments in the
      // loop, which cost it 15 % through spilled registers).
      for (int seg = 0; seg < SEGS; ++seg) {
        if (seg > 0) {
          h = hot(k, at, seg);
          r = part(at, h, seg);
          lds_barrier();  // every wave is past its last fragment read
          fill_first(at, seg, h, r, pt, wu, lane);
        }
        TileFrags<G> f0, f1;
        if (r.n > 0) {
          wait_vmcnt0();
          lds_barrier();
#pragma unroll
          for (int i = 0; i < G::NT; ++i) f0.n[i] = frag_n(sb(0), 0, wn, i, lane);
#pragma unroll
          for (int i = 0; i < G::MT; ++i) f0.m[i] = frag_m(sa(0), 0, wm, i, lane);
        }
        // Per K step i (stage c; the other stages hold the next steps or are
        // filling): slice 0 on f0 while f1 is read; barrier (stage c is free,
        // step i + 1 has landed); slice 1 on f1 while step i + NS is copied into
        // stage c and f0 of step i + 1 is read.
        for (int kt = 0; kt < r.n; kt += G::NS) {
#pragma unroll
          for (int c = 0; c < G::NS; ++c) {
            const int i = kt + c;
            if (i < r.n) {
              const int nx = (c + 1) % G::NS;
              Step st{};
              slice(f0, acc, f1, sa(c), sb(c), 1, wm, wn, lane, false, h, pt, st, c, sa(c), sb(c), wu);
              if (i + 1 < r.n) {
                // the copies of step i + 2 may stay in flight, if that step has
                // any
                if (G::NS > 2 && i + 2 < r.n && (r.s + i + 2) * BK + BK <= h.K)
                  wait_steps<G::NS - 2>();
                else if (EPI != EPI_STORE || G::NS > 2 || i > 0)  // both of two stages have landed before step 0
                  wait_vmcnt0();
                lds_barrier();
              }
              bool cp = false;
              if (i + G::NS < r.n) {
                st = step_at(h, r.s + i + G::NS);
                cp = st.k0 + BK <= h.K;
                if (!cp) tail(k, at, seg, st, sa(c), sb(c), wu, lane);
              }
              slice(f1, acc, f0, sa(nx), sb(nx), 0, wm, wn, lane, cp, h, pt, st, c, sa(c), sb(c), wu);
            }
          }
        }
      }
      lds_barrier();  // every wave is past its last fragment read
      epilogue(k, at, acc, wm, wn, wu, lane, (char*)lds);
      lds_barrier();  // the LDS is free; the stores may still be in flight
      v += gridDim.x;
      if (v >= total) break;
      at = locate(k, v);
      h = hot(k, at, 0);
      r = part(at, h, 0);
      fill_first(at, 0, h, r, pt, wu, lane);
    }
  }
};

template <typename T, typename TO, Lay LA, Lay LB, int SEGS, int EPI, typename G>
__global__ __launch_bounds__(G::THREADS, G::MINW) void tile_kernel(TileOp) {  // read through the argument segment
  __shared__ __attribute__((aligned(1024))) T lds[G::LDS_ELEMS + (G::ROOM ? 0 : 512)];
  Tile<T, TO, LA, LB, SEGS, EPI, G>::run((Args)__builtin_amdgcn_kernarg_segment_ptr(), lds);
}

// Grid: min(#units of work, #CUs x workgroups per CU), the per-CU count from
// the runtime for the compiled kernel, cached per instantiation (atomic:
// concurrent first calls store the same value).
template <typename T, typename TO, Lay LA, Lay LB, int SEGS, int EPI, typename G>
hipError_t launch_tile(TileOp p, hipStream_t stream, int num_cus) {
  p.tiles_m = (p.M + G::BM - 1) / G::BM;
  p.tiles_n = (p.N + G::ON - 1) / G::ON;
  if (p.group_m <= 0) p.group_m = 8;
  static std::atomic<int> per_cu_cache{0};
  int per_cu = per_cu_cache.load(std::memory_order_relaxed);
  if (per_cu == 0) {
    int n = 0;
    hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, tile_kernel<T, TO, LA, LB, SEGS, EPI, G>,
                                                                G::THREADS, 0);
    if (e != hipSuccess) return e;
    per_cu = n > 0 ? n : 1;
    per_cu_cache.store(per_cu, std::memory_order_relaxed);
  }
  const int64_t total = (int64_t)p.tiles_m * p.tiles_n * p.batch * p.splits;
  const int64_t cap = (int64_t)num_cus * per_cu;
  hipLaunchKernelGGL((tile_kernel<T, TO, LA, LB, SEGS, EPI, G>), dim3((unsigned)(total < cap ? total : cap)),
                     dim3(G::THREADS), 0, stream, p);
  return hipGetLastError();
}

}  // namespace
}  // namespace coalesce
