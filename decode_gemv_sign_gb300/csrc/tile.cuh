// Warp-level weight tiles shared by the 4-bit GEMV and the mixture-of-experts
// layer: 16 weight rows by a k-step of columns, brought into shared memory by
// asynchronous copies and multiplied with up to 32 columns of activations on
// BF16 mma.sync tiles (m16n8k16, fp32 accumulation).
//
// At 1..16 rows of x the product does 2..32 operations per weight and streams
// every weight once, so moving the weights is the bound and the warp-level
// MMA is ample: a k-step of 16 x 128 4-bit weights (1 KB) costs 8 MMAs per 8
// columns of x, against about 44 cycles of an SM's share of the HBM rate.
//
// Layout of a 4-bit weight.  Tiles of 16 rows, each a run of blocks of 128
// columns.  A block is 1024 bytes of codes in the MMA's A-fragment order (lane
// l's words at 16 l of each 512-byte half), then 16 x NG scales (NG = 128 / G
// groups per block): word g * NG + j holds the BF16 scales of rows g (low) and
// g + 8 (high) of group j.  Codes and scales of a block are contiguous, so a
// tile is read front to back.  Word 2q + i of lane (g = l / 4, t = l % 4) holds
// the 16 x 4 weights of MMA i of column run q: rows g and g + 8, columns
// c = q4_col(q, t) + 4 i + {0, 1, 2, 3}.  Nibble p (0..3) is the first and
// nibble p + 4 the second column of the MMA's A register p: row g columns c,
// c+1; row g + 8 the same; row g columns c+2, c+3; row g + 8 the same.  So
// (w >> 4p) & 0x000F000F is a pair of codes, which under the exponent of 128
// is the BF16 pair 128 + code; subtracting 136 leaves code - 8 exactly.
//
// Every lane copies the bytes that it will read itself, so a stage needs no
// barrier, only the lane's own cp.async group wait.
#pragma once

#include "wcomp_impl.cuh"

namespace wc {

constexpr int kTileRows = 16;     // weight rows of a tile (the MMA's M side)
constexpr int kQ4Cols = 128;      // columns of a 4-bit block
constexpr int kBfCols = 64;       // columns of a BF16 k-step

__host__ __device__ constexpr uint32_t q4_block_bytes(int ng) { return 1024u + 32u * uint32_t(ng); }

// First of the 8 columns of run q (0..3) that lane t of a quad owns.  Groups
// of 32 columns must not share an MMA, whose sum runs over the quad, so they
// take 32-column runs; wider groups take 16 columns a lane, which x gives in
// one 32-byte load.
template <int NG>
__host__ __device__ constexpr uint32_t q4_col(uint32_t q, uint32_t t) {
  return NG == 4 ? 32 * q + 8 * t : 64 * (q >> 1) + 16 * t + 8 * (q & 1);
}

// ---------------------------------------------------------------------------
// Asynchronous copies and loads.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The same with only the first `bytes` (0..16) read and the rest zero-filled.
__device__ __forceinline__ void cp_async16_part(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds_v2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts_v4(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Activations: 16 or 8 consecutive BF16 values.  CONST: the buffer is not
// written while the kernel runs (read-only path); otherwise a plain load that
// the compiler keeps after the grid barrier that orders it.
template <bool CONST>
__device__ __forceinline__ void ld_x32(const uint16_t* p, uint32_t (&r)[8]) {
  if constexpr (CONST) {
    asm("ld.global.nc.L1::evict_last.v8.u32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "l"(p));
  } else {
    asm volatile("ld.global.v8.u32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p)
                 : "memory");
  }
}
template <bool CONST>
__device__ __forceinline__ void ld_x16(const uint16_t* p, uint32_t* r) {
  if constexpr (CONST) {
    asm("ld.global.nc.L1::evict_last.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "l"(p));
  } else {
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "l"(p)
                 : "memory");
  }
}

// d = a b + d, and d = a b for the first MMA of a chain.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Pair p of a code word as BF16 values code - 8 (exact).
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, int p) {
  uint32_t v = ((w >> (4 * p)) & 0x000F000Fu) | 0x43004300u, d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(0x43084308u));
  return d;
}

// The activations of one lane: a row pointer per 8 columns of x (null: that
// column of x does not exist and counts as zero) and the valid columns of a
// row, a multiple of 16.
template <int NT>
struct XRows {
  const uint16_t* p[NT];
  uint32_t K;
};

// Word w (0..3) of run h (0, 1) of half s: columns q4_col(2 s + h, t) ...
template <int NG, int NT, bool CONST>
__device__ __forceinline__ void load_x_half(const XRows<NT>& x, uint32_t col0, int s, uint32_t t,
                                            uint32_t (&xv)[NT][8]) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 8; ++i) xv[nt][i] = 0u;
    if (!x.p[nt]) continue;
    if constexpr (NG == 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t c = col0 + q4_col<4>(2 * s + h, t);
        if (c < x.K) ld_x16<CONST>(x.p[nt] + c, &xv[nt][4 * h]);
      }
    } else {
      const uint32_t c = col0 + q4_col<1>(2 * s, t);
      if (c < x.K) ld_x32<CONST>(x.p[nt] + c, xv[nt]);
    }
  }
}

// ---------------------------------------------------------------------------
// Sources.  A source says how a tile's k-step reaches its stage and how a
// stage is multiplied; Tile is where one 16-row tile starts.
// ---------------------------------------------------------------------------
template <int NG_>
struct Q4Src {
  static constexpr int NG = NG_;
  static constexpr int kCols = kQ4Cols;
  static constexpr uint32_t kStage = 1024 + 128 * NG;  // every lane keeps its own copy of its two rows' scales
  struct Tile {
    const uint8_t* p;
  };
  static __device__ __forceinline__ void issue(const Tile& tile, uint32_t step, uint32_t st, int lane) {
    const uint8_t* b = tile.p + uint64_t(step) * q4_block_bytes(NG);
    cp_async16(st + lane * 16, b + lane * 16);
    cp_async16(st + 512 + lane * 16, b + 512 + lane * 16);
    cp_async_small<4 * NG>(st + 1024 + lane * 4 * NG, b + 1024 + (lane >> 2) * 4 * NG);
  }
  // MT tiles' stages at st, st + kStage, ... times the step's activations.
  // Codes enter the MMA as exact integers; each group's sum is scaled in fp32.
  template <int MT, int NT, bool CONST>
  static __device__ __forceinline__ void step(uint32_t st, uint32_t stepi, int lane, const XRows<NT>& x,
                                              float (&acc)[MT][NT][4]) {
    const uint32_t t = uint32_t(lane) & 3;
    float ga[MT][NT][4];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t xv[NT][8];
      load_x_half<NG, NT, CONST>(x, stepi * kCols, s, t, xv);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint32_t sm = st + m * kStage;
        const uint4 c4 = lds_v4(sm + s * 512 + lane * 16);
        const uint32_t cw[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // word j: run h = j / 2, MMA j % 2
          const uint32_t a0 = q4_pair(cw[j], 0), a1 = q4_pair(cw[j], 1), a2 = q4_pair(cw[j], 2), a3 = q4_pair(cw[j], 3);
          const bool first = NG == 4 ? (j & 1) == 0 : NG == 2 ? j == 0 : j == 0 && s == 0;
          const bool last = NG == 4 ? (j & 1) == 1 : NG == 2 ? j == 3 : j == 3 && s == 1;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (first)
              mma16816_first(ga[m][nt], a0, a1, a2, a3, xv[nt][2 * j], xv[nt][2 * j + 1]);
            else
              mma16816(ga[m][nt], a0, a1, a2, a3, xv[nt][2 * j], xv[nt][2 * j + 1]);
          }
          if (last) {
            const uint32_t sc = lds_u32(sm + 1024 + lane * 4 * NG + 4 * (NG == 4 ? 2 * s + (j >> 1) : NG == 2 ? s : 0));
            const float sg = bf16_lo(sc), sh = bf16_hi(sc);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              acc[m][nt][0] = fmaf(sg, ga[m][nt][0], acc[m][nt][0]);
              acc[m][nt][1] = fmaf(sg, ga[m][nt][1], acc[m][nt][1]);
              acc[m][nt][2] = fmaf(sh, ga[m][nt][2], acc[m][nt][2]);
              acc[m][nt][3] = fmaf(sh, ga[m][nt][3], acc[m][nt][3]);
            }
          }
        }
      }
    }
  }
};

// Row-major BF16 weights.  VEC: rows of a multiple of 8 columns from a 16-byte
// aligned base, copied asynchronously; otherwise element loads.  A stage holds
// four 512-byte pieces: rows g (pieces 0, 1) and g + 8 (2, 3), columns
// 16 t + 0..7 (even pieces) and + 8..15 (odd pieces) of the step.
template <bool VEC>
struct BfSrc {
  static constexpr int kCols = kBfCols;
  static constexpr uint32_t kStage = 2048;
  struct Tile {
    const uint16_t* p;  // first row of the tile
    uint32_t rows;      // valid rows (0..16)
    uint32_t K;
  };
  static __device__ __forceinline__ void issue(const Tile& tile, uint32_t step, uint32_t st, int lane) {
    const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = g + 8 * (i >> 1), c = step * kCols + 16 * t + 8 * (i & 1);
      const uint16_t* src = tile.p + uint64_t(r) * tile.K + c;
      const uint32_t dst = st + i * 512 + lane * 16;
      if constexpr (VEC) {
        const bool ok = r < tile.rows && c < tile.K;
        cp_async16_part(dst, ok ? src : tile.p, ok ? 16u : 0u);
      } else {
        uint32_t v[4] = {0u, 0u, 0u, 0u};
        if (r < tile.rows)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < tile.K) v[e >> 1] |= uint32_t(__ldg(src + e)) << (16 * (e & 1));
        sts_v4(dst, make_uint4(v[0], v[1], v[2], v[3]));
      }
    }
  }
  template <int MT, int NT, bool CONST>
  static __device__ __forceinline__ void step(uint32_t st, uint32_t stepi, int lane, const XRows<NT>& x,
                                              float (&acc)[MT][NT][4]) {
    const uint32_t t = uint32_t(lane) & 3;
    uint32_t xv[NT][8];
    load_x_half<1, NT, CONST>(x, stepi * kCols, 0, t, xv);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint32_t sm = st + m * kStage + lane * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 wg = lds_v4(sm + h * 512), wh = lds_v4(sm + 1024 + h * 512);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(acc[m][nt], wg.x, wh.x, wg.y, wh.y, xv[nt][4 * h], xv[nt][4 * h + 1]);
          mma16816(acc[m][nt], wg.z, wh.z, wg.w, wh.w, xv[nt][4 * h + 2], xv[nt][4 * h + 3]);
        }
      }
    }
  }
};

// x[B, K] copied to rows of Kp columns (a multiple of 128), zeros past K: for
// an x whose rows do not start on 32-byte boundaries.
__device__ __forceinline__ void pad_rows(const uint16_t* __restrict__ x, uint64_t K, uint64_t Kp, uint32_t B,
                                         uint16_t* __restrict__ out, uint64_t first, uint64_t stride) {
  for (uint64_t i = first; i < uint64_t(B) * Kp; i += stride) {
    const uint64_t b = i / Kp, c = i % Kp;
    out[i] = c < K ? x[b * K + c] : uint16_t(0);
  }
}

}  // namespace wc

// A 4-bit weight: M matrices of N x K, each padded to whole tiles and blocks.
struct wcomp_q4 {
  int64_t M, N, K;
  int group, ng;
  uint64_t tiles, blocks;  // tiles per matrix, blocks per tile
  uint8_t* d = nullptr;
  int device = 0;
  uint64_t matrix_bytes() const { return tiles * blocks * wc::q4_block_bytes(ng); }
};

namespace wc {
// Work counters of the 4-bit and expert kernels on the current device, and
// their error word (defined in q4.cu).  A launch that joins split sums or
// crosses a grid barrier takes a slot of kSlotWords zeroed counters, round
// robin, and leaves them zero.
constexpr uint32_t kSlotWords = 1024;
int work_slot(int dev, uint32_t** slot, uint32_t** err);
}  // namespace wc
