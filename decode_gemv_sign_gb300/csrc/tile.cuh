// Weight tiles shared by the 4-bit GEMV and the mixture-of-experts layer: 32
// weight rows by a k-step of columns, copied to shared memory by TMA and
// multiplied with a few columns of activations on warp-level tensor-core MMAs
// (m16n8k16, fp32 accumulation).
//
// At 1..16 rows of x the product streams every weight once and does little
// with it: moving the weights is the bound, and the multiply has about 44
// cycles of an SM per KB of weights before it falls behind the HBM.
//
// 4-bit weights enter the MMA as exact fp16 integers, by the method published for
// matrix products of 4-bit and fp16 operands: a code under the exponent of 1024 is
// 1024 + c in the low four mantissa bits and 1024 + 16 c in the next four, so a
// word of eight codes takes one shift and four bit operations, and four fused
// multiply-adds on the other pipe leave c - 8.
// (BF16, with 7 mantissa bits, takes three shifts; a BF16 form of the GEMV ran
// at 0.70 of the HBM rate with its integer pipe 55 % busy.  FP8 operands need
// no arithmetic at all, but their warp-level MMA is converted to fp16 again:
// 12 conversions each, slower in all.  Codes as fp16 subnormals need none
// either, but the MMA aligns them by their exponent field and drops bits.)
// The activations are BF16 values brought to fp16 by a power of two per 128
// columns (records, below), which loses nothing down to 2^-31 of the largest.
#pragma once

#include "host_shared.cuh"

namespace wc {

// What a debug build's launches of this translation unit leave out or delay
// (wcomp_debug_skip_first_copy): bit 0 a ring's first copy, bit 1 the first
// block's arrival at a grid barrier.
#if WCOMP_DEBUG
static __device__ uint32_t g_debug_hooks;
#define WCOMP_DEBUG_HOOKS(fn) \
  cudaError_t fn(uint32_t bits) { return cudaMemcpyToSymbol(g_debug_hooks, &bits, sizeof(bits)); }
#else
#define WCOMP_DEBUG_HOOKS(fn) \
  cudaError_t fn(uint32_t) { return cudaSuccess; }
#endif

constexpr int kTileRows = 32;    // rows of a tile: two MMAs' M side
constexpr int kQ4Cols = 256;     // columns of a 4-bit block
constexpr int kSub = 128;        // columns of half a block, and of an x record
constexpr int kBfCols = 64;      // columns of a BF16 k-step

// A 4-bit block is 32 rows x 256 columns: 4096 bytes of codes, then the scales
// (NG = 128 / group groups per half).  Codes: for half s, 16-row half-tile m
// and quarter q, lane l's 16 bytes at ((2 s + m) 2 + q) 512 + 16 l: the words
// of the MMAs i = 4 q .. 4 q + 3.  Lane (g = l / 4, t = l % 4) holds in the
// word of MMA i the columns c .. c + 3, c = 32 (i / 2) + 8 t + 4 (i % 2): bytes
// 0 and 2 are row g, bytes 1 and 3 row g + 8, columns c, c + 1 (low and high
// nibble) in the first and c + 2, c + 3 in the second.  Scales: the word at
// 4096 + 4 (((s NG + j) 2 + m) 8 + g) has the BF16 scales of rows g (low half)
// and g + 8 of group j.  Sizes are multiples of 128 bytes: copies of 1056-byte
// blocks ran at 0.62-0.8 of the HBM rate, of aligned ones at 0.94.
__host__ __device__ constexpr uint32_t q4_block_bytes(int ng) { return 4096u + 128u * uint32_t(ng); }
__host__ __device__ constexpr uint32_t q4_scale_at(int ng, uint32_t s, uint32_t j, uint32_t m, uint32_t g) {
  return 4096u + 4u * (((s * uint32_t(ng) + j) * 2u + m) * 8u + g);
}

// ---------------------------------------------------------------------------
// Copies, barriers, loads.
// ---------------------------------------------------------------------------
constexpr uint64_t kCopyNs = 1000000000ull;  // how long a wait for copies may take (1 s)

__device__ __forceinline__ uint64_t timer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void bar_init(uint32_t bar) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_passed(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Wait for a phase; false if kCopyNs went by without it.
__device__ __forceinline__ bool bar_wait_long(uint32_t bar, uint32_t parity) {
  const uint64_t deadline = timer_ns() + kCopyNs;
  while (!bar_passed(bar, parity))
    if (timer_ns() > deadline) return false;
  return true;
}
// `bytes` (a multiple of 16) contiguous bytes to shared memory, counted on bar.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// A box of a 2-D tensor map at column c (a multiple of 8 BF16 values), row r.
__device__ __forceinline__ void box_copy(uint32_t dst, const CUtensorMap* map, uint32_t c, uint32_t r, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(r), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint4 lds_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
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
// 32 bytes from a 32-byte boundary.  Not the read-only path: activations may
// be written by the same kernel, before a grid barrier.
__device__ __forceinline__ void ldg_v8(const void* p, uint32_t (&r)[8]) {
  asm volatile("ld.global.v8.u32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ float ldg_f(const void* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
// d = a b + d: BF16, 16 x 16 times 16 x 8.
__device__ __forceinline__ void mma_bf16_k16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same in fp16, and its first of a chain.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// The MMA's A registers of a code word.  `magic` is the exponent pattern
// 0x64006400 in a register the compiler cannot see through: with both patterns
// as immediates each bit operation takes two instructions, on the pipe that
// bounds the multiply.
__device__ __forceinline__ uint32_t q4_magic() { return 0x64006400u | threadIdx.y; }  // blocks are one-dimensional
__device__ __forceinline__ void q4_operand(uint32_t w, uint32_t magic, uint32_t (&a)[4]) {
  const uint32_t w8 = w >> 8;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(a[0]) : "r"(w), "n"(0x000F000F), "r"(magic));
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(a[1]) : "r"(w8), "n"(0x000F000F), "r"(magic));
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(a[2]) : "r"(w), "n"(0x00F000F0), "r"(magic));
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(a[3]) : "r"(w8), "n"(0x00F000F0), "r"(magic));
  // (1024 + c) - 1032 and (1024 + 16 c) / 16 - 72
#pragma unroll
  for (int i = 0; i < 2; ++i) asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(a[i]) : "r"(0x64086408u));
#pragma unroll
  for (int i = 2; i < 4; ++i) asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(a[i]) : "r"(0x2C002C00u), "r"(0xD480D480u));
}

// ---------------------------------------------------------------------------
// Activations for 4-bit weights.  128 values of one row become a record of 256
// bytes: fp16 values under a power of two that brings the largest magnitude (of
// all 128, or of each 32) to [2^14, 2^15), and its inverse, the factor, in a
// separate array.  A BF16 value that is at least 2^-31 of that magnitude keeps
// all its bits; what is smaller errs by less than 2^-39 of it, far below what
// fp32 sums of the record keep.  MMA i's operand of columns c .. c + 3 (see the
// block's layout) is (x[c], x[c + 2]), (x[c + 1], x[c + 3]) at 128 (i / 4) + 32
// t + 8 (i % 4).  An infinity or a NaN keeps its place (finite values beside it
// lose bits, in sums that are not finite).
//
// Factors: NF per record, [record][NF][pitch] with one column per row of
// activations, so that the rows' factors of a record share a line or two: NF =
// 1 and pitch 16 for the layer's input, NF = 4 (each 32 values) and pitch 256
// for the experts' hidden values.
// ---------------------------------------------------------------------------
constexpr uint32_t kRecord = 256;
template <int NF>
constexpr uint32_t factor_pitch() { return NF == 1 ? 16 : 256; }

// The scaling of values whose largest magnitude has the bits m.
__device__ __forceinline__ int record_exponent(uint32_t m) {
  const int k = 14 - (int(m >> 23) - 127);
  return m == 0u ? 0 : k > 120 ? 120 : k;
}
__device__ __forceinline__ float power_of_two(int k) { return __uint_as_float(uint32_t(127 + k) << 23); }
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// One record of BF16 values by one warp: lane l gives columns 4 l .. 4 l + 3.
__device__ __forceinline__ void record_store(uint8_t* rec, float* factor, const float (&v)[4], int lane) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = __reduce_max_sync(0xffffffffu, m);
  const int k = record_exponent(m);
  const float up = power_of_two(k);
  const uint32_t i = (uint32_t(lane) >> 3) * 2 + (uint32_t(lane) & 1), t = (uint32_t(lane) & 7) >> 1;
  *reinterpret_cast<uint2*>(rec + (i >> 2) * 128 + t * 32 + (i & 3) * 8) =
      make_uint2(half2_bits(v[0] * up, v[2] * up), half2_bits(v[1] * up, v[3] * up));
  if (lane == 0) *factor = power_of_two(-k);
}

// One warp's product with R rows of activations in TILES column tiles of the
// MMA: row b is column b % 8 of tile b / 8.  Columns of rows that do not exist
// read one that does; the MMA keeps columns apart and those sums are not used.
template <int TILES>
struct XRows {
  const uint8_t* x[TILES];      // this lane's column, at its 32 bytes of a record
  const float* f[TILES][2];     // the factors of the rows of this lane's two accumulator columns
};
// row(b): first record of row b (of R); column(b): its column of the factors.
template <int TILES, class ROW, class COLUMN>
__device__ __forceinline__ XRows<TILES> x_rows(uint32_t R, int lane, ROW row, COLUMN column) {
  const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
  auto pick = [&](uint32_t b) { return b < R ? b : 0; };
  XRows<TILES> x;
#pragma unroll
  for (int n = 0; n < TILES; ++n) {
    x.x[n] = row(pick(8 * n + g)) + t * 32;
    x.f[n][0] = column(pick(8 * n + 2 * t));
    x.f[n][1] = column(pick(8 * n + 2 * t + 1));
  }
  return x;
}

// 64 columns of every row, from byte `at` of the rows.  SHARED: x's records and
// factors are in shared memory.
template <int TILES, bool SHARED = false>
struct XQuarter {
  uint32_t b[TILES][8];
  __device__ __forceinline__ void load(const XRows<TILES>& x, uint64_t at) {
#pragma unroll
    for (int n = 0; n < TILES; ++n) {
      if constexpr (SHARED) {
        const uint4* p = reinterpret_cast<const uint4*>(x.x[n] + uint32_t(at));
        const uint4 lo = p[0], hi = p[1];
        b[n][0] = lo.x; b[n][1] = lo.y; b[n][2] = lo.z; b[n][3] = lo.w;
        b[n][4] = hi.x; b[n][5] = hi.y; b[n][6] = hi.z; b[n][7] = hi.w;
      } else {
        ldg_v8(x.x[n] + at, b[n]);
      }
    }
  }
};
template <int TILES, int NF, bool SHARED = false>
struct XFactors {
  float f[TILES][2][NF];
  __device__ __forceinline__ void load(const XRows<TILES>& x, uint32_t rec) {
    const uint64_t at = uint64_t(rec) * (NF * factor_pitch<NF>());
#pragma unroll
    for (int n = 0; n < TILES; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const float* p = x.f[n][i] + at + j * factor_pitch<NF>();
          f[n][i][j] = SHARED ? *p : ldg_f(p);
        }
  }
};

// ---------------------------------------------------------------------------
// Sources: how a tile's k-step reaches its stage, and a stage its product.  A
// Cursor is a place in one tile.
// ---------------------------------------------------------------------------
template <int NG_>
struct Q4Src {
  static constexpr int NG = NG_;
  static constexpr int kCols = kQ4Cols;
  static constexpr uint32_t kStage = q4_block_bytes(NG);
  static constexpr bool kCopies = true;
  struct Cursor {
    const uint8_t* p;
  };
  // K-step `step` of tile `tile` of a matrix at m whose tiles have `steps`.
  static __device__ __forceinline__ Cursor at(const uint8_t* m, uint32_t steps, uint32_t tile, uint32_t step) {
    return {m + (uint64_t(tile) * steps + step) * kStage};
  }
  // Copy the cursor's block to the stage and move on to the next (one lane).
  static __device__ __forceinline__ void issue(Cursor& c, uint32_t st, uint32_t bar) {
    bulk_copy(st, c.p, kStage, bar);
    c.p += kStage;
  }
  // Quarter q of half s of a stage times x.  Columns with one scale and one
  // factor are summed in ga by the MMAs; the sum enters acc under scale times
  // factor.  That product, of 8 bits and a power of two, comes first: it is exact,
  // while the sum times one of the two alone may pass fp32's range although the
  // result does not (scales of 2^110 with x of 2^-100).
  template <int TILES, int NF, bool SHARED>
  static __device__ __forceinline__ void quarter(uint32_t st, uint32_t s, int q, int lane, uint32_t magic,
                                                 const XQuarter<TILES, SHARED>& x,
                                                 const XFactors<TILES, NF, SHARED>& f,
                                                 float (&ga)[2][TILES][4], float (&acc)[2][TILES][4]) {
    constexpr int RUNS = NG > NF ? NG : NF;    // runs per half: 8 / RUNS MMAs each
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint4 w4 = lds_v4(st + s * 2048 + (m * 2 + q) * 512 + lane * 16);
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
      float sg = 1.f, sh = 1.f;
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        const int i = 4 * q + ii;
        uint32_t a[4];
        q4_operand(w[ii], magic, a);
#pragma unroll
        for (int n = 0; n < TILES; ++n) {
          if ((i * RUNS) % 8 == 0)
            mma_f16_first(ga[m][n], a, x.b[n][2 * ii], x.b[n][2 * ii + 1]);
          else
            mma_f16(ga[m][n], a, x.b[n][2 * ii], x.b[n][2 * ii + 1]);
        }
        if (((i + 1) * RUNS) % 8 != 0) continue;
        if (NG > 2 || RUNS == 1 || ii + 1 == 8 / RUNS) {  // a quarter has one scale a row, or (NG = 4) two
          const uint32_t sc = lds_u32(st + q4_scale_at(NG, 0, i * NG / 8, m, 0) + s * (64 * NG) + (lane >> 2) * 4);
          sg = bf16_lo(sc);
          sh = bf16_hi(sc);
        }
#pragma unroll
        for (int n = 0; n < TILES; ++n)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[m][n][v] = fmaf((v < 2 ? sg : sh) * f.f[n][v & 1][i * NF / 8], ga[m][n][v], acc[m][n][v]);
      }
    }
  }
};

// Row-major BF16 weights, viewed as one matrix of rows (all experts').  A box may
// reach past its expert's last row into the next one's: MMA rows do not mix, and
// the sums of those are not used.
//
// MAP: rows of a multiple of 8 columns from a 16-byte aligned base, copied as
// boxes of 32 rows x 64 columns through a tensor map (zeros past the last
// column and row), whose 128-byte swizzle puts 16-byte chunk c of row r at
// chunk c ^ (r % 8): the lanes' reads meet no bank conflict.
template <bool MAP>
struct BfSrc {
  static constexpr int NG = 0;
  static constexpr int kCols = kBfCols;
  static constexpr uint32_t kStage = 4096;
  static constexpr bool kCopies = true;
  struct Cursor {
    const CUtensorMap* map;
    uint32_t row, col;  // first row of the tile, first column of the step
  };
  static __device__ __forceinline__ Cursor at(const CUtensorMap* map, const uint16_t*, uint64_t, uint64_t row, uint32_t,
                                              uint32_t col) {
    return {map, uint32_t(row), col};
  }
  static __device__ __forceinline__ void issue(Cursor& c, uint32_t st, uint32_t bar) {
    box_copy(st, c.map, c.col, c.row, bar);
    c.col += kCols;
  }
  // A stage times x: lane (g, t) holds columns 16 t .. 16 t + 15 of rows g,
  // g + 8, ... and the same columns of its row of x.
  template <int NT>
  static __device__ __forceinline__ void multiply(uint32_t st, int lane, const XQuarter<NT>& x,
                                                  float (&acc)[2][NT][4]) {
    const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint32_t sm = st + m * 2048 + g * 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = sm + (((2 * t + h) ^ g) << 4);  // rows g and g + 8 have the same swizzle
        const uint4 wg = lds_v4(at), wh = lds_v4(at + 1024);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_bf16_k16(acc[m][nt], wg.x, wh.x, wg.y, wh.y, x.b[nt][4 * h], x.b[nt][4 * h + 1]);
          mma_bf16_k16(acc[m][nt], wg.z, wh.z, wg.w, wh.w, x.b[nt][4 * h + 2], x.b[nt][4 * h + 3]);
        }
      }
    }
  }
};

// Any row length and any 2-byte aligned base, in 4-byte asynchronous copies: row
// r's stage has the 33 words that cover its 64 columns from the word boundary at
// or before the first, a lane a word, at a pitch of 33 words, so that the lanes'
// reads (eight words of their own, and the one after) meet no bank conflict.
// After the rows stand the number of columns left to their end and which rows
// start in the middle of a word: the reader undoes that, and clears in the stage
// what lies past the rows' end.
// (us with element loads / with both undone word by word / so: 15 tokens, 4 of 14
// experts of 2014 x 1556: 321 / 118 / 97; 5 tokens, 3 of 12 of 1001 x 333: - / 33 /
// 26, where 1000 x 328 takes 19 through boxes.)
template <>
struct BfSrc<false> {
  static constexpr int NG = 0;
  static constexpr int kCols = kBfCols;
  static constexpr uint32_t kPitch = 132, kMarks = 32 * kPitch, kStage = kMarks + 16;
  static constexpr bool kCopies = false;
  struct Cursor {
    const uint16_t* w;    // the matrix
    uint64_t rows, row;   // its rows; the first of the tile
    uint32_t K, col;
  };
  static __device__ __forceinline__ Cursor at(const CUtensorMap*, const uint16_t* w, uint64_t rows, uint64_t row,
                                              uint32_t K, uint32_t col) {
    return {w, rows, row, K, col};
  }
  // 4 bytes, of which `bytes` (0, 2 or 4) are read and the rest zero.
  static __device__ __forceinline__ void copy4(uint32_t dst, uint64_t src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  }
  static __device__ __forceinline__ void load(Cursor& c, uint32_t st, int lane) {
    const uint64_t row = 2 * uint64_t(c.K), base = reinterpret_cast<uint64_t>(c.w), end = base + c.rows * row;
    const uint64_t at = base + c.row * row + 2 * c.col, mine = at + lane * row;
    auto word_of = [](uint64_t a) { return a & ~uint64_t(3); };
    if (lane == 0)
      asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(st + kMarks), "r"(c.K - c.col),
                   "r"((uint32_t(at >> 1) & 1u) | (c.K & 1u) << 1)
                   : "memory");
    // rows whose 33 words lie in the matrix, and the others that it has
    const bool inside = word_of(mine) >= base && mine + 132 <= end;
    const uint32_t rows = __ballot_sync(0xffffffffu, inside);
    uint32_t rest = __ballot_sync(0xffffffffu, !inside && c.row + lane < c.rows);
    if (inside) copy4(st + lane * kPitch + 128, word_of(mine) + 128, 4u);
    const uint32_t dst = st + lane * 4;
    uint64_t even = word_of(at) + 4 * lane, odd = word_of(at + row) + 4 * lane;  // two rows are whole words
#pragma unroll
    for (int r = 0; r < 32; r += 2, even += 2 * row, odd += 2 * row) {
      if (rows >> r & 1) copy4(dst + r * kPitch, even, 4u);
      if (rows >> r & 2) copy4(dst + (r + 1) * kPitch, odd, 4u);
    }
    // at the matrix's ends: each word as far as it lies in it
#pragma unroll 1
    for (; rest; rest &= rest - 1) {
      const uint32_t r = __ffs(rest) - 1;
#pragma unroll 1
      for (uint32_t i = lane; i < 33; i += 32) {
        const uint64_t a = word_of(at + r * row) + 4 * i;
        const uint32_t to = st + r * kPitch + i * 4;
        if (a >= base)
          copy4(to, a < end ? a : word_of(base) + 4, a >= end ? 0u : end - a < 4 ? uint32_t(end - a) : 4u);
        else  // the first word of an unaligned matrix: its upper half
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(uint32_t(c.w[0]) << 16) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    c.col += kCols;
  }
  template <int NT>
  static __device__ __forceinline__ void multiply(uint32_t st, int lane, const XQuarter<NT>& x,
                                                  float (&acc)[2][NT][4]) {
    const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
    const uint32_t cols = lds_u32(st + kMarks), marks = lds_u32(st + kMarks + 4);
    auto odd = [&](uint32_t r) { return (marks ^ (marks >> 1 & r)) & 1u; };  // row r starts in mid-word
    if (cols < kBfCols) {
      const uint32_t row = st + lane * kPitch, h = cols + odd(lane);
      if (h & 1) asm volatile("st.shared.u16 [%0], %1;" ::"r"(row + h * 2), "h"(uint16_t(0)) : "memory");
#pragma unroll 1
      for (uint32_t i = (h + 1) >> 1; i < 33; ++i)
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(row + i * 4), "r"(0u) : "memory");
      __syncwarp();
    }
    const uint32_t shift = odd(g) * 16;  // rows 8 apart start alike
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint32_t sm = st + (16 * m + g) * kPitch + t * 32;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a[2][5];  // rows g and g + 8: four words and the one after
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < 5; ++i) a[r][i] = lds_u32(sm + r * 8 * kPitch + (4 * h + i) * 4);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) a[r][i] = __funnelshift_r(a[r][i], a[r][i + 1], shift);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_bf16_k16(acc[m][nt], a[0][0], a[1][0], a[0][1], a[1][1], x.b[nt][4 * h], x.b[nt][4 * h + 1]);
          mma_bf16_k16(acc[m][nt], a[0][2], a[1][2], a[0][3], a[1][3], x.b[nt][4 * h + 2], x.b[nt][4 * h + 3]);
        }
      }
    }
  }
};

// One warp's ring of D stages, and the mbarrier of each.  `left` counts the
// copies in flight.  A wait that runs out sets the error word and marks the
// ring dead once what is in flight has had its time to land: no more copies
// and waits, and the sums go on with whatever the stages hold.
template <class SRC, int D>
struct Ring {
  uint32_t base, bars;
  uint32_t* err;
  uint32_t slot = 0, parity = 0, left = 0;
  bool dead = false;
#if WCOMP_DEBUG
  bool skip = g_debug_hooks & 1u;  // the first copy is left out
#else
  static constexpr bool skip = false;
#endif

  __device__ __forceinline__ Ring(uint32_t base_, uint32_t bars_, uint32_t* err_, int lane)
      : base(base_), bars(bars_), err(err_) {
    if (lane < D) bar_init(bars + 8 * lane);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
  }
  __device__ __forceinline__ uint32_t stage() const { return base + slot * SRC::kStage; }
  // Refill slot `at` with the cursor's next k-step.
  __device__ __forceinline__ void refill(uint32_t at, typename SRC::Cursor& c, int lane) {
    const uint32_t st = base + at * SRC::kStage;
    if constexpr (SRC::kCopies) {
      if (dead) return;
      if (lane == 0 && !skip) {
        bar_expect(bars + 8 * at, SRC::kStage);
        SRC::issue(c, st, bars + 8 * at);
      }
#if WCOMP_DEBUG
      skip = false;
#endif
      ++left;
    } else {
      SRC::load(c, st, lane);
      ++left;
    }
  }
  __device__ __forceinline__ void wait(int lane) {
    if constexpr (SRC::kCopies) {
      if (!dead) {
        bool ok = bar_passed(bars + 8 * slot, parity);
        if (!__all_sync(0xffffffffu, ok)) {
          if (!ok) ok = bar_wait_long(bars + 8 * slot, parity);
          if (!__all_sync(0xffffffffu, ok)) give_up(lane);
        }
        --left;
      }
    } else {
      // the lanes' copies in groups: the oldest of D, or all of fewer
      if (left == D)
        asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
      else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      --left;
      __syncwarp();
    }
  }
  __device__ __forceinline__ void give_up(int lane) {
    dead = true;
    if (lane == 0) atomicOr(err, 1u);
    uint32_t s = slot, q = parity;
    for (uint32_t i = 0; i < left; ++i) {
      bar_wait_long(bars + 8 * s, q);
      if (++s == D) {
        s = 0;
        q ^= 1;
      }
    }
    __syncwarp();
  }
  // Let what is in flight land without using it.
  __device__ __forceinline__ void abandon() {
    if constexpr (!SRC::kCopies) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (!dead) {
      dead = true;
      for (; left; --left) {
        bar_wait_long(bars + 8 * slot, parity);
        next();
      }
    }
  }
  __device__ __forceinline__ void next() {
    if (++slot == D) {
      slot = 0;
      parity ^= 1;
    }
  }
};

// A warp's product of ring stages with its activations, one k-step after the
// other: begin(k) loads the first activations, step(k, kn) multiplies the
// ring's current stage, which holds k-step k, adds to acc, refills the slot by
// issue(slot) with the copy cursor's next k-step and moves on; kn is the
// k-step of the stage after it.  Activations are loaded 64 columns ahead of
// their use, factors 128: their latency (L2's, for a first touch) would
// otherwise stand in every step.
template <class SRC, int TILES, int NF, bool SHARED = false>
struct Product {  // 4-bit
  XQuarter<TILES, SHARED> x0;
  XFactors<TILES, NF, SHARED> f;
  __device__ __forceinline__ void begin(const XRows<TILES>& x, uint32_t k) {
    if (TILES == 1 || NF == 1) f.load(x, 2 * k);
    x0.load(x, uint64_t(2 * k) * kRecord);
  }
  template <class RING, class ISSUE>
  __device__ __forceinline__ void step(RING& ring, uint32_t k, uint32_t kn, int lane, uint32_t magic,
                                       const XRows<TILES>& x, float (&acc)[2][TILES][4], ISSUE& issue) {
    const uint32_t st = ring.stage();
    ring.wait(lane);
    // unrolled, where registers allow, for the scheduler to find independent
    // work: a warp's own chain of dependencies is what bounds a step (us rolled /
    // unrolled: 16384 x 53248, B = 1 78.9 / 76.0, 8 83.1 / 79.4; two tiles, which spill: 111 / 117)
#pragma unroll (TILES == 1 ? 2 : 1)
    for (uint32_t s = 0; s < 2; ++s) {
      const uint32_t rec = 2 * k + s, next = s ? 2 * kn : rec + 1;
      float ga[2][TILES][4];
      XQuarter<TILES, SHARED> x1;
      XFactors<TILES, NF, SHARED> fn;
      constexpr bool kAhead = TILES == 1 || NF == 1;  // sixteen rows' four factors: no registers left to load ahead
      x1.load(x, uint64_t(rec) * kRecord + 128);
      if (kAhead)
        fn.load(x, next);
      else
        f.load(x, rec);
      SRC::template quarter<TILES, NF, SHARED>(st, s, 0, lane, magic, x0, f, ga, acc);
      x0.load(x, uint64_t(next) * kRecord);
      SRC::template quarter<TILES, NF, SHARED>(st, s, 1, lane, magic, x1, f, ga, acc);
      if (kAhead) f = fn;
    }
    __syncwarp();  // every lane has read the stage
    issue(ring.slot);
    ring.next();
  }
};
template <bool MAP, int TILES, int NF>
struct Product<BfSrc<MAP>, TILES, NF, false> {
  XQuarter<TILES> x0;
  __device__ __forceinline__ void begin(const XRows<TILES>& x, uint32_t k) { x0.load(x, uint64_t(k) * (2 * kBfCols)); }
  template <class RING, class ISSUE>
  __device__ __forceinline__ void step(RING& ring, uint32_t, uint32_t kn, int lane, uint32_t, const XRows<TILES>& x,
                                       float (&acc)[2][TILES][4], ISSUE& issue) {
    const uint32_t st = ring.stage();
    XQuarter<TILES> x1;
    if (TILES < 4) x1.load(x, uint64_t(kn) * (2 * kBfCols));
    ring.wait(lane);
    BfSrc<MAP>::multiply(st, lane, x0, acc);
    __syncwarp();
    issue(ring.slot);
    ring.next();
    if (TILES < 4)
      x0 = x1;
    else
      x0.load(x, uint64_t(kn) * (2 * kBfCols));
  }
};

template <int N>
__device__ __forceinline__ void zero(float (&acc)[2][N][4]) {
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < N; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
}
// A warp's accumulators to its place in shared memory, [half-tile][TILES][lane][4].
template <int N>
__device__ __forceinline__ void put_sums(float* part, int lane, const float (&acc)[2][N][4]) {
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < N; ++n)
      *reinterpret_cast<float4*>(part + (m * N + n) * 128 + lane * 4) =
          make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
}

// Row r (0..31) of a tile, column b: the sum over `warps` warps' accumulators,
// [half-tile][TILES][lane][4] each and `stride` floats apart, in their order.
template <int TILES>
__device__ __forceinline__ float warp_sums(const float* part, int warps, uint32_t stride, uint32_t r, uint32_t b) {
  const uint32_t m = r >> 4, j = r & 15;
  const float* p = part + (m * TILES + (b >> 3)) * 128 + (j & 7) * 16 + ((b & 7) >> 1) * 4 + (j >> 3) * 2 + (b & 1);
  float v = 0.f;
  for (int w = 0; w < warps; ++w) v += p[w * stride];
  return v;
}

// ---------------------------------------------------------------------------
// Cutting work over the CTAs.  `units` units of `steps` k-steps each stand in
// one row; CTA c takes k-steps [start(c), start(c + 1)).  With `split` the cuts
// fall anywhere, so every CTA streams the same bytes; otherwise on whole units.
// The part of a cut unit that a CTA holds goes to the workspace, and the CTA
// that arrives last at the unit's counter adds the parts in the order of the
// CTAs: the result does not depend on which one that is.  Or, where there are few
// units, each is shared by a `team` of CTAs (a cluster), the k-steps evenly.
// ---------------------------------------------------------------------------
constexpr uint32_t kJoinCopies = 24;  // what a join of gate and up parts costs, in 4 KB copies of a CTA
__host__ __device__ __forceinline__ uint32_t cdiv32(uint32_t a, uint32_t b) { return (a + b - 1) / b; }
struct Cuts {
  uint32_t units, steps, split, team = 1;
  uint32_t grid;        // CTAs that have work, at most one per k-step (split) or unit
  uint32_t quot, rem;   // pieces (k-steps or units) per CTA; the first rem CTAs take one more
  // Cut units anywhere where that shortens the longest CTA's run by more than a
  // join costs, in k-steps.  Work is cut by k-steps only below 2^32 of them, so
  // that 32-bit divisions do (a 64-bit one takes most of a microsecond, and
  // several would stand before the first copy of a phase).
  __host__ __device__ Cuts(uint32_t units_, uint32_t steps_, uint32_t ctas, uint32_t join) : units(units_), steps(steps_) {
    const uint64_t all = uint64_t(units) * steps;
    const uint32_t rounds = cdiv32(units, ctas);
    split = (all >> 31) == 0 && uint64_t(rounds) * steps > cdiv32(uint32_t(all), ctas) + join;
    const uint32_t work = split ? uint32_t(all) : units;
    grid = work < ctas ? work : ctas;
    quot = work / grid;
    rem = work - quot * grid;
  }
  // First piece of CTA c.
  __device__ __forceinline__ uint32_t start(uint32_t c) const { return quot * c + (c < rem ? c : rem); }
  // The CTA that has k-step s (split only).
  __device__ __forceinline__ uint32_t owner(uint32_t s) const {
    const uint32_t big = (quot + 1) * rem;
    return s < big ? s / (quot + 1) : rem + (s - big) / quot;
  }
};

// The units' parts of this CTA's range, one after the other: part [k0, k1) of
// `unit`, and a warp's share [w0, w1) of it.
struct Parts {
  uint32_t steps, unit, k0, k1, left;
  __device__ __forceinline__ explicit Parts(const Cuts& c, bool teams = false) : steps(c.steps) {
    if (teams) {  // one part, of at least one k-step
      unit = blockIdx.x / c.team;
      const uint32_t rank = blockIdx.x - unit * c.team;
      k0 = steps * rank / c.team;
      k1 = steps * (rank + 1) / c.team;
      left = k1 - k0;
      return;
    }
    const uint32_t cta = blockIdx.x < c.grid ? blockIdx.x : c.grid, begin = c.start(cta);
    const uint32_t pieces = blockIdx.x < c.grid ? c.start(cta + 1) - begin : 0u;
    unit = c.split ? begin / c.steps : begin;
    k0 = c.split ? begin - unit * c.steps : 0u;
    left = c.split ? pieces : pieces * c.steps;  // k-steps, of 4 KB: never 2^32 of them
    cut();
  }
  __device__ __forceinline__ void cut() { k1 = left < steps - k0 ? k0 + left : steps; }
  __device__ __forceinline__ bool more() const { return left != 0; }
  __device__ __forceinline__ bool whole() const { return k0 == 0 && k1 == steps; }
  __device__ __forceinline__ void next() {
    left -= k1 - k0;
    ++unit;
    k0 = 0;
    cut();
  }
  __device__ __forceinline__ uint32_t w0(uint32_t warp) const { return k0 + share(warp); }
  __device__ __forceinline__ uint32_t w1(uint32_t warp) const { return k0 + share(warp + 1); }
  // len * i / 8 without overflow (8 warps share a part)
  __device__ __forceinline__ uint32_t share(uint32_t i) const {
    const uint32_t len = k1 - k0;
    return (len >> 3) * i + (((len & 7) * i) >> 3);
  }
};

// This CTA's part of a cut unit, n floats given by value(i), joined with the
// others'; store(i, sum) runs in the last CTA to arrive.  part: 2 n_max floats
// per CTA; counters: one per CTA, zero before and after.  All threads call it.
template <class VALUE, class STORE>
__device__ __forceinline__ void join_parts(const Cuts& c, const Parts& s, bool first_part, float* part, uint32_t n_max,
                                           uint32_t* counters, uint32_t n, uint32_t* s_flag, VALUE value, STORE store) {
  const uint32_t g0 = s.unit * c.steps;
  float* mine = part + (2 * uint64_t(blockIdx.x) + (first_part ? 0 : 1)) * n_max;
  for (uint32_t i = threadIdx.x; i < n; i += blockDim.x) __stcg(mine + i, value(i));
  const uint32_t first = c.owner(g0), last = c.owner(g0 + c.steps - 1);
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    *s_flag = atomicAdd(counters + first, 1u) == last - first;
    __threadfence();
  }
  __syncthreads();
  if (!*s_flag) return;
  // the first CTA's range may have begun before the unit, which it then keeps second
  const float* head = part + (2 * uint64_t(first) + (c.start(first) < g0 ? 1 : 0)) * n_max;
  const float* rest = part + 2 * uint64_t(first + 1) * n_max;
  for (uint32_t i = threadIdx.x; i < n; i += blockDim.x) {
    float v = __ldcg(head + i);
#pragma unroll 1
    for (uint32_t q0 = 0; q0 < last - first; q0 += 16) {  // 16 loads in flight
      float t[16];
#pragma unroll
      for (uint32_t q = 0; q < 16; ++q)
        t[q] = q0 + q < last - first ? __ldcg(rest + 2 * uint64_t(q0 + q) * n_max + i) : 0.f;
#pragma unroll
      for (uint32_t q = 0; q < 16; ++q) v += t[q];
    }
    store(i, v);
  }
  if (threadIdx.x == 0) counters[first] = 0u;
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
// The 4-bit and expert kernels' error word on device `dev`, and kSlotWords zero
// counters for a launch on stream s that crosses grid barriers, which it leaves
// zero: the stream's, or, for a launch that is captured, a set of its own as long
// as its graph is there, since it may run next to any other as often as that
// does.  Null when those are used up: the caller clears counters of its own in
// front of the launch.  Defined in q4.cu.
constexpr uint32_t kSlotWords = 1024;
int work_error(int dev, uint32_t** err);
int work_slot(int dev, cudaStream_t s, uint32_t** slot);
}  // namespace wc
