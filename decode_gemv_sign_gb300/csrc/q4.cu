// Weights in 4 bits with group scales: quantise, read back, and the
// matrix-vector product y[B, N] = x[B, K] . W^T for 1..16 rows of x.
//
//   s[r, j] = bf16(max |w| / 7) over the G columns of group j of row r,
//   c[r, k] = clamp(rint(w / s), -7, 7) + 8,    value (c - 8) s,
//   y[b, r] = sum_j s[r, j] sum_{k in j} (c[r, k] - 8) x[b, k].
#include <string.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <new>

#include "tile.cuh"

namespace wc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ---------------------------------------------------------------------------
// Quantise, read back, and the plain layouts.  One warp takes a quarter block
// (16 rows x 128 columns: half s, 16-row half-tile m); lane (g, t) holds the 32
// columns 32 q + 8 t .. + 7 (run q = 0..3) of rows g and g + 8, so codes leave
// in the operands' order with no exchange, and a group's largest magnitude
// needs two shuffles in a quad.
// ---------------------------------------------------------------------------
// A CTA takes a run of 8 x `run` quarter blocks of one tile, so that what needs
// a division is found once for all of them.
struct Blocks {
  uint8_t* d;
  uint64_t N, K, tiles, blocks;
  uint64_t runs;         // M * tiles * runs_per_tile
  uint32_t runs_per_tile, run;
};

// A quarter block: its block, place in it, first row and column in its matrix,
// and that row's index over all matrices.
struct At {
  uint64_t block, r0, k0, row;
  uint32_t s, m;
};
// f(quarter) for this warp's quarter blocks of every run of its CTA.
template <class F>
__device__ __forceinline__ void each_quarter(const Blocks& b, F f) {
  for (uint64_t run = blockIdx.x; run < b.runs; run += gridDim.x) {
    const uint64_t tile = run / b.runs_per_tile, mat = tile / b.tiles;
    const uint32_t first = uint32_t(run - tile * b.runs_per_tile) * (kWarps * b.run), end = uint32_t(b.blocks) * 4;
    const uint64_t r0 = (tile - mat * b.tiles) * kTileRows;
#pragma unroll 1
    for (uint32_t j = 0; j < b.run; ++j) {
      const uint32_t q = first + j * kWarps + (threadIdx.x >> 5);
      if (q >= end) break;
      At a;
      a.s = (q >> 1) & 1;
      a.m = q & 1;
      a.block = tile * b.blocks + (q >> 2);
      a.r0 = r0 + 16 * a.m;
      a.k0 = uint64_t(q >> 2) * kQ4Cols + kSub * a.s;
      a.row = mat * b.N + a.r0;
      f(a);
    }
  }
}
__device__ __forceinline__ uint8_t* codes_at(uint8_t* block, const At& a, int lane) {
  return block + (2 * a.s + a.m) * 1024 + lane * 16;
}

// Larger magnitudes (NaN if there is one), with a sign that means nothing.
__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The BF16 scale of a group whose largest magnitude (BF16 bits, NaN if it
// holds one) is m: the nearest BF16 to m / 7.  m has 8 significant bits, so
// m / 7 is never nearer than 2^-12 of itself to a midpoint of two BF16 values,
// and the rounding of 1 / 7 and of the product cannot cross it.  A group with
// an infinity or a NaN gets the scale NaN.
__device__ __forceinline__ uint32_t scale_of(uint32_t m) {
  uint16_t s;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(s) : "f"(__fmul_rn(__uint_as_float(m << 16), 1.f / 7.f)));
  return m >= 0x7F80u ? 0x7FC0u : s;
}

// Code of one weight.  w / s has a quotient of 8-bit significands: it is
// either exactly halfway between integers or at least 2^-10 away from it, so
// w * (1 / s) (2^-22 relative error), rounded to a multiple of 2^-12 by the
// first constant, is on the right side of every halfway point, and exactly on
// it where w / s is; the second constant then rounds half to even.  Scales
// below 2^-100 (reciprocals near overflow, quotients above 7) divide and clamp.
constexpr float kSnap = 3072.f;        // 1.5 * 2^11: ulp 2^-12
// Codes come as kBase + code, so that a word of eight is a sum of them times
// powers of 16, less what the bases add up to: one integer multiply-add a code.
constexpr float kRound = 12582920.f;   // 1.5 * 2^23 + 8: ulp 1, and the code's offset of 8
constexpr uint32_t kBase = 0x4B400000u;  // the bits of 1.5 * 2^23
__device__ __forceinline__ uint32_t code_fast(float w, float rs) {
  return __float_as_uint(__fadd_rn(__fadd_rn(__fmaf_rn(w, rs, kSnap), -kSnap), kRound));
}
__device__ __forceinline__ uint32_t code_slow(float w, float s) {
  if (!(s > 0.f)) return 8u;  // scale 0 or NaN
  return uint32_t(int(fminf(fmaxf(rintf(__fdiv_rn(w, s)), -7.f), 7.f)) + 8);
}

// 8 columns of row r from column c as BF16 pairs; zeros outside the matrix.
__device__ __forceinline__ void load8(const uint16_t* __restrict__ row, uint64_t c, uint64_t K, bool ok, uint32_t* v) {
  uint4 q = make_uint4(0u, 0u, 0u, 0u);
  if (ok && c < K) q = ld_stream_v4(row + c);
  v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
}

// Rows that start anywhere (K % 8 != 0, or an unaligned tensor) pass through
// shared memory, a warp's 16 x 128 values at kPitch: in memory a warp then
// touches 64 consecutive bytes at a time instead of 2 bytes in each of 32
// places (5001 x 7003: quantise 51 -> 25 us, read back 134 -> 18 us).
constexpr uint32_t kPitch = 136;
__device__ __forceinline__ void rows_in(const uint16_t* __restrict__ w, const At& a, const Blocks& b, uint16_t* tile,
                                        int lane) {
#pragma unroll 4
  for (uint32_t r = 0; r < 16; ++r) {
    const bool ok = a.r0 + r < b.N;
    const uint16_t* row = w + (a.row + r) * b.K + a.k0;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t c = lane + 32 * i;
      tile[r * kPitch + c] = ok && a.k0 + c < b.K ? __ldg(row + c) : uint16_t(0);
    }
  }
}
__device__ __forceinline__ void rows_out(uint16_t* __restrict__ out, const At& a, const Blocks& b, const uint16_t* tile,
                                         int lane) {
#pragma unroll 4
  for (uint32_t r = 0; r < 16; ++r) {
    if (a.r0 + r >= b.N) break;
    uint16_t* row = out + (a.row + r) * b.K + a.k0;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t c = lane + 32 * i;
      if (a.k0 + c < b.K) row[c] = tile[r * kPitch + c];
    }
  }
}

// Codes and scales of one quarter block to memory: columns 2 e and 2 e + 1 of
// run q are a byte (low and high nibble) of word 2 q + e / 2, at bit 16 (e % 2)
// for row g and 8 above it for row g + 8.
template <int NG>
__device__ __forceinline__ void store_quarter(uint8_t* block, const At& a, int lane, const uint32_t (&words)[8],
                                              const uint32_t (&sc)[2][NG]) {
  uint8_t* out = codes_at(block, a, lane);
  *reinterpret_cast<uint4*>(out) = make_uint4(words[0], words[1], words[2], words[3]);
  *reinterpret_cast<uint4*>(out + 512) = make_uint4(words[4], words[5], words[6], words[7]);
  const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
  if (int(t) < NG) {  // lane t of a quad writes group t's scales
    uint32_t s2 = sc[0][0] | (sc[1][0] << 16);
#pragma unroll
    for (int j = 1; j < NG; ++j)
      if (int(t) == j) s2 = sc[0][j] | (sc[1][j] << 16);
    *reinterpret_cast<uint32_t*>(block + q4_scale_at(NG, a.s, t, a.m, g)) = s2;
  }
}

__device__ __forceinline__ float reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// The codes of a quarter block with a scale that code_fast does not take, from
// the weights and the stored scales again: rare, and kept apart from the
// kernel's registers and instruction cache.
template <int NG>
__device__ __noinline__ void slow_codes(const uint16_t* __restrict__ w, uint64_t K, uint32_t rows, uint64_t k0,
                                        uint8_t* block, uint32_t s, uint32_t m, int lane) {
  const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
#pragma unroll 1
  for (uint32_t j = 0; j < 8; ++j) {
    uint32_t word = 0u;
#pragma unroll 1
    for (uint32_t n = 0; n < 8; ++n) {  // nibble n: column 2 (n / 4) + n % 2 of four, row half n / 2 % 2
      const uint32_t r = (n >> 1) & 1;
      const uint64_t c = k0 + 32 * (j >> 1) + 8 * t + 4 * (j & 1) + 2 * (n >> 2) + (n & 1);
      uint32_t code = 8u;
      if (g + 8 * r < rows && c < K) {
        const uint32_t sc = *reinterpret_cast<const volatile uint32_t*>(block + q4_scale_at(NG, s, (j >> 1) * NG / 4, m, g));
        code = code_slow(__uint_as_float(uint32_t(w[uint64_t(g + 8 * r) * K + c]) << 16), r ? bf16_hi(sc) : bf16_lo(sc));
      }
      word |= code << (4 * n);
    }
    *reinterpret_cast<uint32_t*>(block + (2 * s + m) * 1024 + (j >> 2) * 512 + lane * 16 + (j & 3) * 4) = word;
  }
}

template <int NG, bool VEC>
__global__ void __launch_bounds__(kThreads) q4_encode_kernel(const uint16_t* __restrict__ w,
                                                             const __grid_constant__ Blocks b) {
  __shared__ __align__(16) uint16_t tiles[VEC ? 1 : kWarps * 16 * kPitch];
  const int lane = threadIdx.x & 31;
  const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
  each_quarter(b, [&](const At& a) {
    uint32_t v[2][4][4];  // row half, run, pairs
    uint16_t* tile = tiles + (VEC ? 0 : (threadIdx.x >> 5) * 16 * kPitch);
    if (!VEC) {
      __syncwarp();
      rows_in(w, a, b, tile, lane);
      __syncwarp();
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool ok = a.r0 + g + 8 * r < b.N;
      const uint16_t* row = w + (a.row + g + 8 * r) * b.K;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (VEC) {
          load8(row, a.k0 + 32 * q + 8 * t, b.K, ok, v[r][q]);
        } else {
          const uint4 u = *reinterpret_cast<const uint4*>(tile + (g + 8 * r) * kPitch + 32 * q + 8 * t);
          v[r][q][0] = u.x; v[r][q][1] = u.y; v[r][q][2] = u.z; v[r][q][3] = u.w;
        }
      }
    }
    uint32_t sc[2][NG];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        uint32_t m = 0u;
#pragma unroll
        for (int q = j * 4 / NG; q < (j + 1) * 4 / NG; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) m = abs_max2(m, v[r][q][e]);
        m = abs_max2(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = abs_max2(m, __shfl_xor_sync(0xffffffffu, m, 2));
        m = abs_max2(m, m >> 16) & 0x7FFFu;
        sc[r][j] = scale_of(m);
      }
    float rs[2][NG];
    bool slow = false;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const float s = __uint_as_float(sc[r][j] << 16);
        const bool fast = s >= 0x1p-100f;
        slow |= !fast && s != 0.f;
        rs[r][j] = fast ? reciprocal(s) : 0.f;  // scale 0: every code is 8
      }
    uint32_t words[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) words[j] = 0u - kBase * 0x11111111u;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          words[2 * q + (e >> 1)] += code_fast(bf16_lo(v[r][q][e]), rs[r][q * NG / 4]) * (1u << (16 * (e & 1) + 8 * r)) +
                                     code_fast(bf16_hi(v[r][q][e]), rs[r][q * NG / 4]) * (16u << (16 * (e & 1) + 8 * r));
    uint8_t* block = b.d + a.block * q4_block_bytes(NG);
    store_quarter<NG>(block, a, lane, words, sc);
    if (__any_sync(0xffffffffu, slow)) {
      __syncwarp();
      slow_codes<NG>(w + a.row * b.K, b.K, uint32_t(a.r0 < b.N ? (b.N - a.r0 < 16 ? b.N - a.r0 : 16) : 0), a.k0, block,
                     a.s, a.m, lane);
    }
  });
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// (c - 8) * s is an integer of at most 4 bits times an 8-bit significand: the
// BF16 multiply rounds the exact product once.  c | 0x4300 is the BF16 value
// 128 + c, so taking 136 away leaves c - 8 exactly.
template <int NG, bool VEC>
__global__ void __launch_bounds__(kThreads) q4_decode_kernel(const __grid_constant__ Blocks b,
                                                             uint16_t* __restrict__ out) {
  __shared__ __align__(16) uint16_t tiles[VEC ? 1 : kWarps * 16 * kPitch];
  const int lane = threadIdx.x & 31;
  const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
  uint16_t* tile = tiles + (VEC ? 0 : (threadIdx.x >> 5) * 16 * kPitch);
  each_quarter(b, [&](const At& a) {
    uint8_t* block = b.d + a.block * q4_block_bytes(NG);
    const uint8_t* in = codes_at(block, a, lane);
    const uint4 c0 = ld_stream_v4(in), c1 = ld_stream_v4(in + 512);
    const uint32_t cw[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    uint32_t sc[NG];
#pragma unroll
    for (int j = 0; j < NG; ++j) sc[j] = ld_stream_u32(block + q4_scale_at(NG, a.s, j, a.m, g));
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (VEC && a.r0 + g + 8 * r >= b.N) continue;
      uint16_t* row = out + (a.row + g + 8 * r) * b.K;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t s2 = prmt(sc[q * NG / 4], 0u, r ? 0x3232u : 0x1010u);
        uint32_t v[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // columns 0, 2 and 1, 3 of the word as pairs, then in order
          const uint32_t w = cw[2 * q + e] >> (8 * r);
          uint32_t even, odd;
          asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(even) : "r"((w & 0x000F000Fu) | 0x43004300u), "r"(0x43084308u));
          asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(odd) : "r"(((w >> 4) & 0x000F000Fu) | 0x43004300u), "r"(0x43084308u));
          even = mul2(even, s2);
          odd = mul2(odd, s2);
          v[2 * e] = prmt(even, odd, 0x5410u);
          v[2 * e + 1] = prmt(even, odd, 0x7632u);
        }
        const uint64_t c = a.k0 + 32 * q + 8 * t;
        if constexpr (VEC) {
          if (c < b.K) *reinterpret_cast<uint4*>(row + c) = make_uint4(v[0], v[1], v[2], v[3]);
        } else {
          *reinterpret_cast<uint4*>(tile + (g + 8 * r) * kPitch + 32 * q + 8 * t) = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
    }
    if (!VEC) {
      __syncwarp();
      rows_out(out, a, b, tile, lane);
      __syncwarp();
    }
  });
}

// Plain layout to blocks and back.  Plain codes: row r's ceil(K / 2) bytes,
// column 2j in the low nibble of byte j; plain scales: BF16 [rows, ceil(K/G)].
// Columns past K and rows past N become code 8 with scale 0.
template <int NG>
__global__ void __launch_bounds__(kThreads) q4_pack_kernel(const uint8_t* __restrict__ codes,
                                                           const uint16_t* __restrict__ scales,
                                                           const __grid_constant__ Blocks b) {
  const int lane = threadIdx.x & 31;
  const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
  const uint64_t pitch = (b.K + 1) / 2, groups = cdiv(b.K, kSub / NG);
  each_quarter(b, [&](const At& a) {
    uint32_t words[8], sc[2][NG];
#pragma unroll
    for (int j = 0; j < 8; ++j) words[j] = 0u;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool ok = a.r0 + g + 8 * r < b.N;
      const uint8_t* row = codes + (a.row + g + 8 * r) * pitch;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint64_t c = a.k0 + 32 * q + 8 * t;
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // columns c + 2 e, c + 2 e + 1
          uint32_t lo = 8u, hi = 8u;
          if (ok && c + 2 * e < b.K) {
            const uint32_t byte = row[(c >> 1) + e];
            lo = byte & 15u;
            if (c + 2 * e + 1 < b.K) hi = byte >> 4;
          }
          words[2 * q + (e >> 1)] |= (lo | (hi << 4)) << (16 * (e & 1) + 8 * r);
        }
      }
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const uint64_t gr = a.k0 / (kSub / NG) + j;
        sc[r][j] = ok && gr < groups ? uint32_t(scales[(a.row + g + 8 * r) * groups + gr]) : 0u;
      }
    }
    store_quarter<NG>(b.d + a.block * q4_block_bytes(NG), a, lane, words, sc);
  });
}

template <int NG>
__global__ void __launch_bounds__(kThreads) q4_unpack_kernel(const __grid_constant__ Blocks b,
                                                             uint8_t* __restrict__ codes,
                                                             uint16_t* __restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
  const uint64_t pitch = (b.K + 1) / 2, groups = cdiv(b.K, kSub / NG);
  each_quarter(b, [&](const At& a) {
    uint8_t* block = b.d + a.block * q4_block_bytes(NG);
    const uint8_t* in = codes_at(block, a, lane);
    const uint4 c0 = ld_stream_v4(in), c1 = ld_stream_v4(in + 512);
    const uint32_t cw[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (a.r0 + g + 8 * r >= b.N) continue;
      uint8_t* row = codes + (a.row + g + 8 * r) * pitch;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint64_t c = a.k0 + 32 * q + 8 * t;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (c + 2 * e < b.K) row[(c >> 1) + e] = uint8_t(cw[2 * q + (e >> 1)] >> (16 * (e & 1) + 8 * r));
        }
      }
      const uint64_t gr = a.k0 / (kSub / NG) + t;
      if (int(t) < NG && gr < groups)
        scales[(a.row + g + 8 * r) * groups + gr] =
            uint16_t(ld_stream_u32(block + q4_scale_at(NG, a.s, t, a.m, g)) >> (16 * r));
    }
  });
}

// ---------------------------------------------------------------------------
// GEMV.  x becomes records (record_store): where they are few, in every block's
// shared memory, while its first weights are on their way; otherwise by a kernel
// of their own, before the end of which the GEMV is launched, to fill its rings
// with weights and only then wait for the records.  A unit is a tile of 32 rows,
// whose k-steps the warps of a CTA share; the units' k-steps fall on the CTAs as
// plan() says.
//
// Measured on 16384 x 53248 (450 MB at groups of 128: 66 us at the rate of a
// plain copy): 76 us for one row of x (0.87 of that rate), 77 for 4, 79.5 for
// 8, 111 for 16; 90 and 133 for 8 and 16 rows at groups of 32 (73 us).  Up to 8
// rows what is left is the start, the joins (5 us together) and each warp's chain
// through some 120 instructions per KB, two thirds of them the codes' expansion: a
// k-step takes a warp 1.0 us with 8 warps on half of the SMs, 1.6 with 16 on all,
// with rings of any depth.  At 16 rows no unit is over half busy (tensor cores 43 %):
// the latency of twice the MMAs with the 16 warps that 128 registers leave an SM.
// x is not it (with all of it in one line of L1 the time does not fall), nor are
// more warps (10 or 12 of a CTA spill).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) q4_x_kernel(const uint16_t* __restrict__ x, uint64_t K, uint32_t recs, uint32_t B,
                                                   uint8_t* __restrict__ out, float* __restrict__ factors,
                                                   uint32_t* __restrict__ counters, uint32_t n_counters) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0)  // the joins' counters, for after the GEMV's wait
    for (uint32_t j = threadIdx.x; j < n_counters; j += blockDim.x) counters[j] = 0u;
  const int lane = threadIdx.x & 31;
  const uint64_t i = uint64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (i >= uint64_t(B) * recs) return;
  const uint64_t b = i / recs, k = (i - b * recs) * kSub + 4 * lane;
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = k + e < K ? __uint_as_float(uint32_t(x[b * K + k + e]) << 16) : 0.f;
  record_store(out + i * kRecord, factors + (i - b * recs) * factor_pitch<1>() + b, v, lane);
}

struct GemvArgs {
  const uint8_t* w;
  const uint16_t* x;    // records in shared memory: x[B, K]
  uint64_t K;
  const uint8_t* xq;    // records in memory: [B][2 * steps]
  const float* factors;
  float* y;
  float* part;          // 2 B rows-of-a-unit floats per CTA
  uint32_t* counters;   // one per CTA, zero at the first join
  uint32_t* err;
  uint64_t N;
  Cuts cuts{1, 1, 1, 0};
  int B;
};

constexpr int kDepth = 2;  // stages of a warp: a third takes L1 from the activations (16384 x 53248, B = 16: 111 -> 130 us)

// Records in shared memory: at most eight a warp, rows 16 bytes further apart
// than their records, for the banks, then the factors.  For up to 8 rows of x
// and one part of a unit a block.  us on the GPU / on the host for a kernel of
// its own, and so: 2048 x 6144 6.0 / 7.6, 5.4 / 4.5; 1024 x 4096 4.6 / 7.8, 4.3 /
// 4.3; 6144 x 6144 8.8 / 7.1, 8.8 / 4.4; 2048 x 16384 in clusters 8.6 / 7.4, 8.8 /
// 4.4; with more units than blocks it lost 0.7 us on the GPU (16384 x 6144).
constexpr uint32_t kXRecords = 8 * kWarps;
constexpr uint32_t kXShared = kXRecords * (kRecord + 16 + factor_pitch<1>() * 4);

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A float of the cluster's CTA `rank` at the place that `a` has in this one.
__device__ __forceinline__ float cluster_lds(uint32_t a, uint32_t rank) {
  float v;
  asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\tld.shared::cluster.f32 %0, [r];\n\t}"
               : "=f"(v)
               : "r"(a), "r"(rank)
               : "memory");
  return v;
}

template <int NG, int TILES, bool SHARED>
constexpr uint32_t q4_smem() {
  return kWarps * (kDepth * Q4Src<NG>::kStage + 2 * TILES * 512 + kDepth * 8) + 128 + (SHARED ? kXShared : 0);
}

// SHARED: x's records in shared memory; TEAM: a unit is shared by a cluster.
template <int NG, int TILES, bool SHARED, bool TEAM>
__global__ void __launch_bounds__(kThreads, 2) q4_gemv_kernel(const __grid_constant__ GemvArgs p) {
  using S = Q4Src<NG>;
  const uint32_t magic = q4_magic();
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 127u);
  float* part = reinterpret_cast<float*>(smem + kWarps * kDepth * S::kStage);  // [warp][half-tile][TILES][lane][4]
  __shared__ uint32_t s_flag;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Ring<S, kDepth> ring(smem_u32(smem) + uint32_t(warp) * kDepth * S::kStage,
                       smem_u32(part + kWarps * 2 * TILES * 128) + uint32_t(warp) * kDepth * 8, p.err, lane);
  // The copy cursor runs kDepth k-steps ahead of the sums, across units.
  Parts ahead(p.cuts, TEAM);
  const uint32_t r0 = SHARED ? 2 * ahead.k0 : 0;  // first record of x
  const uint32_t recs = SHARED ? 2 * (ahead.k1 - ahead.k0) : 2 * p.cuts.steps;
  uint32_t ileft = 0;
  typename S::Cursor it{};
  auto enter = [&]() {
    for (; ahead.more(); ahead.next()) {
      const uint32_t w0 = ahead.w0(warp), w1 = ahead.w1(warp);
      if (w0 == w1) continue;
      ileft = w1 - w0;
      it = S::at(p.w, p.cuts.steps, ahead.unit, w0);
      ahead.next();
      return;
    }
  };
  auto issue = [&](uint32_t slot) {
    if (ileft) {
      ring.refill(slot, it, lane);
      if (--ileft == 0) enter();
    }
  };
  enter();
#pragma unroll
  for (int i = 0; i < kDepth; ++i) issue(i);
  // records in shared memory, or from memory
  uint8_t* const xs = reinterpret_cast<uint8_t*>(part + kWarps * 2 * TILES * 128) + kWarps * kDepth * 8;
  const uint64_t pitch = SHARED ? recs * kRecord + 16 : recs * uint64_t(kRecord);
  const uint8_t* const rows = SHARED ? xs : p.xq;
  float* const fs = reinterpret_cast<float*>(xs + p.B * pitch);
  const float* const factors = SHARED ? fs : p.factors;
  if constexpr (SHARED) {
    const uint32_t n = p.B * recs;
    const bool words = p.K % 4 == 0 && (reinterpret_cast<uintptr_t>(p.x) & 7) == 0;
    uint2 v[8];  // all of a warp's records in flight
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t i = warp + j * kWarps, b = i / recs, k = (r0 + i - b * recs) * kSub + 4 * lane;
      const uint16_t* from = p.x + uint64_t(b) * p.K + k;
      v[j] = make_uint2(0u, 0u);
      if (i < n && k < p.K) {
        if (words) {
          v[j] = *reinterpret_cast<const uint2*>(from);
        } else {
          const uint32_t left = uint32_t(p.K) - k;
          v[j].x = from[0] | (left > 1 ? uint32_t(from[1]) << 16 : 0u);
          v[j].y = (left > 2 ? uint32_t(from[2]) : 0u) | (left > 3 ? uint32_t(from[3]) << 16 : 0u);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t i = warp + j * kWarps, b = i / recs, rec = i - b * recs;
      if (i < n) {
        const float f[4] = {bf16_lo(v[j].x), bf16_hi(v[j].x), bf16_lo(v[j].y), bf16_hi(v[j].y)};
        record_store(xs + b * pitch + rec * kRecord, fs + rec * factor_pitch<1>() + b, f, lane);
      }
    }
    __syncthreads();
  }
  const XRows<TILES> x =
      x_rows<TILES>(uint32_t(p.B), lane, [&](uint32_t b) { return rows + b * pitch - r0 * kRecord; },
                    [&](uint32_t b) { return factors + b - r0 * factor_pitch<1>(); });
  if constexpr (!SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");  // the records are there
  const uint32_t outs = kTileRows * p.B;
  bool first_part = true;
  for (Parts s(p.cuts, TEAM); s.more(); s.next(), first_part = false) {
    const uint32_t w0 = s.w0(warp), w1 = s.w1(warp);
    float acc[2][TILES][4];
    zero<TILES>(acc);
    if (w0 < w1) {
      Product<S, TILES, 1, SHARED> prod;
      prod.begin(x, w0);
      for (uint32_t k = w0; k < w1; ++k) prod.step(ring, k, k + 1 < w1 ? k + 1 : k, lane, magic, x, acc, issue);
    }
    __syncthreads();  // the previous unit's parts are read
    put_sums<TILES>(part + warp * 2 * TILES * 128, lane, acc);
    __syncthreads();
    // output o: row o % 32 of the tile, batch row o / 32; the warps in order
    auto value = [&](uint32_t o) { return warp_sums<TILES>(part, kWarps, 2 * TILES * 128, o % kTileRows, o / kTileRows); };
    auto store = [&](uint32_t o, float v) {
      const uint64_t r = uint64_t(s.unit) * kTileRows + o % kTileRows;
      if (r < p.N) p.y[uint64_t(o / kTileRows) * p.N + r] = v;
    };
    if constexpr (TEAM) {  // the only part: the rings are idle, and their place takes its sums
      float* const mine = reinterpret_cast<float*>(smem);
      for (uint32_t o = threadIdx.x; o < outs; o += kThreads) mine[o] = value(o);
      cluster_sync();
      if (blockIdx.x == s.unit * p.cuts.team)  // the first CTA adds all, in their order
        for (uint32_t o = threadIdx.x; o < outs; o += kThreads) {
          float v = mine[o];
          for (uint32_t r = 1; r < p.cuts.team; ++r) v += cluster_lds(smem_u32(mine + o), r);
          store(o, v);
        }
      cluster_sync();  // they are read
    } else if (s.whole()) {
      for (uint32_t o = threadIdx.x; o < outs; o += kThreads) store(o, value(o));
    } else {
      join_parts(p.cuts, s, first_part, p.part, outs, p.counters, outs, &s_flag, value, store);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// Sets of counters: one for each of kStreams streams, whose launches follow one
// another, then those of captured launches.  (Sets in turn for launches on any
// stream would be shared by two that run together when one stream is that many
// launches ahead.)  The first kKept captured launches keep theirs for good; the
// next take kLent more, which come back with their graph.  What a graph holds for
// that costs each of its launches 2.3 us and 0.14 us a call (2 of 8 experts of 1024
// x 512 as a graph of one call, 16.9 -> 19.2 us), too much for the few graphs that
// most programs make once, and less than clearing counters in the graph, 4 us a
// call.
constexpr uint64_t kStreams = StreamNumbers::kStreams, kKept = 1024, kLent = 4096;
std::mutex g_mu;
struct Work {
  uint32_t* err = nullptr;
  uint32_t* sets = nullptr;
  uint32_t taken = 0;         // of the captured launches' sets, how many were ever taken
  uint32_t back = 0;          // lent ones that came back
  uint16_t returned[kLent];
  StreamNumbers streams;
} g_work[64];

// Zeroed memory at *p, allocated on first use.
int first_use(uint32_t** p, size_t bytes) {
  return *p ? int(WCOMP_OK) : map_cuda(zeroed_alloc(p, bytes));
}

template <int NG, int TILES, bool SHARED, bool TEAM>
int prepare_gemv(int dev) {
  static std::atomic<int> cache[64];
  int per_sm = cache[dev].load(std::memory_order_acquire);
  if (!per_sm) {
    auto kern = q4_gemv_kernel<NG, TILES, SHARED, TEAM>;
    constexpr uint32_t smem = q4_smem<NG, TILES, SHARED>();
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess) return -1;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, smem) != cudaSuccess ||
        per_sm < 1)
      return -1;
    cache[dev].store(per_sm, std::memory_order_release);
  }
  return per_sm;
}

template <int NG, int TILES, bool SHARED, bool TEAM>
int launch_gemv(GemvArgs& p, int dev, cudaStream_t s) {
  if (prepare_gemv<NG, TILES, SHARED, TEAM>(dev) < 0) return map_cuda(cudaGetLastError());
  int st = work_error(dev, &p.err);
  if (st != WCOMP_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.cuts.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = q4_smem<NG, TILES, SHARED>();
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if constexpr (TEAM) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = p.cuts.team;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if constexpr (SHARED) {
    const cudaError_t e = cudaLaunchKernelEx(&cfg, q4_gemv_kernel<NG, TILES, SHARED, TEAM>, p);
    count_launches(1);
    return map_cuda(e);
  } else {
    const uint32_t recs = 2 * p.cuts.steps;
    const uint64_t b_xq = uint64_t(p.B) * recs * kRecord, b_f = (recs * factor_pitch<1>() * 4 + 255) & ~uint64_t(255);
    const uint64_t b_part = p.cuts.split ? uint64_t(2) * p.cuts.grid * p.B * kTileRows * sizeof(float) : 0;
    const uint32_t n_counters = p.cuts.split ? p.cuts.grid : 0;
    uint8_t* ws = nullptr;
    cudaError_t e = pool_alloc(reinterpret_cast<void**>(&ws), b_xq + b_f + b_part + n_counters * sizeof(uint32_t), s);
    if (e != cudaSuccess) return map_cuda(e);
    p.xq = ws;
    float* factors = reinterpret_cast<float*>(ws + b_xq);
    p.factors = factors;
    p.part = reinterpret_cast<float*>(ws + b_xq + b_f);
    p.counters = reinterpret_cast<uint32_t*>(ws + b_xq + b_f + b_part);
    q4_x_kernel<<<uint32_t(cdiv(uint64_t(p.B) * recs, 8)), 256, 0, s>>>(p.x, p.K, recs, uint32_t(p.B), ws, factors,
                                                                       p.counters, n_counters);
    e = cudaGetLastError();
    if (e == cudaSuccess) {
      attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
      ++cfg.numAttrs;
      e = cudaLaunchKernelEx(&cfg, q4_gemv_kernel<NG, TILES, SHARED, TEAM>, p);
      count_launches(2);
    }
    cudaFreeAsync(ws, s);
    return map_cuda(e);
  }
}

// How the units' k-steps fall on the CTAs: whole, cut anywhere and joined
// through memory, or shared by clusters of 2 to 8 and joined through shared
// memory: by the longest CTA's run in k-steps, eight of which its warps take at
// once, in 1 us where half of the SMs have work and 1.6 where all have, and by what
// else each costs: a cut some 5 us on a half-filled GPU (2048 x 6144: 16 k-steps
// fewer, 3.7 us longer) and 3 on a full one (6144 x 16384: 16 fewer, 0.6 longer).
// us whole / cut / shared by clusters: 2048 x 6144 5.3 / 9.0 / 5.4; 4096 x 4096, 8
// rows 6.1 / 11.3 / 7.0; 512 x 8192, 3 rows 6.9 / 6.4 / 5.0; 2048 x 16384 10.7 / 11.7 /
// 8.8, 16 rows 15.8 / 16.4 / 12.0; 256 x 40576, 7 rows 24.9 / 10.0 / 7.7; 6144 x 16384,
// 4 rows 17.7 / 18.3 / -; 16384 x 6144 14.2 / 17.7 / -; 16384 x 53248 82 / 76 / -.
constexpr uint32_t kCutCost = 40, kTeamCost = 16;  // k-steps
constexpr uint32_t kXCost = 8;                     // the kernel for x
bool x_shared(const Cuts& c, int B, uint32_t ctas) {  // one part a CTA, of few records
  return B <= 8 && !c.split && c.units <= ctas && uint64_t(B) * 2 * cdiv32(c.steps, c.team) <= kXRecords;
}
Cuts plan(uint32_t units, uint32_t steps, int B, uint32_t ctas) {
  auto at_once = [](uint64_t k) { return cdiv(k, kWarps) * kWarps; };
  Cuts best(units, steps, ctas, kCutCost);
  uint64_t cost = best.split ? at_once(cdiv(uint64_t(units) * steps, ctas)) + kCutCost
                             : at_once(steps) * cdiv32(units, ctas);
  cost += x_shared(best, B, ctas) ? 0 : kXCost;
  for (uint32_t team = 2; team <= 8 && team <= steps && uint64_t(units) * team <= ctas; team *= 2) {
    Cuts c = best;
    c.team = team;
    c.split = 0;
    c.grid = units * team;
    const uint64_t with = at_once(cdiv32(steps, team)) + kTeamCost + (x_shared(c, B, ctas) ? 0 : kXCost);
    if (with < cost) {
      cost = with;
      best = c;
    }
  }
  return best;
}

template <int NG>
int dispatch_gemv(GemvArgs& p, int dev, cudaStream_t s) {
  const int per_sm = p.B <= 8 ? prepare_gemv<NG, 1, false, false>(dev) : prepare_gemv<NG, 2, false, false>(dev);
  if (per_sm < 0) return map_cuda(cudaGetLastError());
  const uint32_t ctas = uint32_t(per_sm * sm_count(dev));
  p.cuts = plan(p.cuts.units, p.cuts.steps, p.B, ctas);
  if (p.B > 8)
    return p.cuts.team > 1 ? launch_gemv<NG, 2, false, true>(p, dev, s) : launch_gemv<NG, 2, false, false>(p, dev, s);
  if (p.cuts.team > 1)
    return x_shared(p.cuts, p.B, ctas) ? launch_gemv<NG, 1, true, true>(p, dev, s)
                                       : launch_gemv<NG, 1, false, true>(p, dev, s);
  return x_shared(p.cuts, p.B, ctas) ? launch_gemv<NG, 1, true, false>(p, dev, s)
                                     : launch_gemv<NG, 1, false, false>(p, dev, s);
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int shape_ok(int64_t M, int64_t N, int64_t K, int group) {
  if (M <= 0 || N <= 0 || K <= 0 || (group != 32 && group != 64 && group != 128)) return WCOMP_EINVAL;
  if (K >= (int64_t(1) << 31) || N >= (int64_t(1) << 31) || M >= (int64_t(1) << 31)) return WCOMP_EUNSUPPORTED;
  // bytes of the held form, with room to spare in 64 bits
  if (double(M) * double(N + 16) * double(K + 128) > 0x1p60) return WCOMP_EUNSUPPORTED;
  if (cdiv(uint64_t(N), kTileRows) * uint64_t(M) >= (uint64_t(1) << 31)) return WCOMP_EUNSUPPORTED;
  return WCOMP_OK;
}

int make_q4(int64_t M, int64_t N, int64_t K, int group, cudaStream_t s, wcomp_q4** out) {
  wcomp_q4* c = new (std::nothrow) wcomp_q4;
  if (!c) return WCOMP_ENOMEM;
  c->M = M;
  c->N = N;
  c->K = K;
  c->group = group;
  c->ng = kSub / group;
  c->tiles = cdiv(uint64_t(N), kTileRows);
  c->blocks = cdiv(uint64_t(K), kQ4Cols);
  cudaGetDevice(&c->device);
  const cudaError_t e = pool_alloc(reinterpret_cast<void**>(&c->d), uint64_t(M) * c->matrix_bytes(), s);
  if (e != cudaSuccess) {
    delete c;
    return map_cuda(e);
  }
  *out = c;
  return WCOMP_OK;
}

// `most`: the longest run, where that still leaves 16 CTAs per SM (quantising
// gains from runs of 8, reading back from none)
Blocks blocks_of(const wcomp_q4* c, uint32_t most) {
  const uint64_t ctas = cdiv(uint64_t(c->M) * c->tiles * c->blocks * 4, kWarps);
  const uint32_t run = uint32_t(std::max<uint64_t>(1, std::min<uint64_t>(most, ctas / (uint64_t(sm_count(c->device)) * 16))));
  const uint32_t per = uint32_t(cdiv(c->blocks * 4, kWarps * run));
  return {c->d, uint64_t(c->N), uint64_t(c->K), c->tiles, c->blocks, uint64_t(c->M) * c->tiles * per, per, run};
}

uint32_t block_grid(const Blocks& b) {
  return uint32_t(std::min<uint64_t>(b.runs, uint64_t(1) << 30));
}

bool on_device(const wcomp_q4* c) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == c->device;
}

}  // namespace

int work_error(int dev, uint32_t** err) {
  if (dev < 0 || dev >= 64) return WCOMP_EUNSUPPORTED;
  std::lock_guard<std::mutex> g(g_mu);
  const int st = first_use(&g_work[dev].err, 128);
  *err = g_work[dev].err;
  return st;
}

namespace {

// A lent set comes back: the destructor of the object that its graphs hold, run
// when the last of them is gone and its last launch has finished.  The object's
// pointer is the device and the set.
void CUDART_CB give_back(void* object) {
  const uintptr_t v = reinterpret_cast<uintptr_t>(object);
  std::lock_guard<std::mutex> g(g_mu);
  Work& w = g_work[v / kLent];
  w.returned[w.back++] = uint16_t(v % kLent);
}

// A set for a launch captured in `graph`; null if there is none left.
uint32_t* captured_set(int dev, cudaGraph_t graph) {
  Work& w = g_work[dev];
  uint32_t* const first = w.sets + kStreams * kSlotWords;
  uint64_t lent;
  {
    std::lock_guard<std::mutex> g(g_mu);
    if (w.taken < kKept) return first + w.taken++ * kSlotWords;
    if (w.back)
      lent = w.returned[--w.back];
    else if (w.taken < kKept + kLent)
      lent = w.taken++ - kKept;
    else
      return nullptr;
  }
  void* const object = reinterpret_cast<void*>(uintptr_t(dev) * kLent + lent);
  cudaUserObject_t o = nullptr;
  if (cudaUserObjectCreate(&o, object, give_back, 1, cudaUserObjectNoDestructorSync) != cudaSuccess) {
    cudaGetLastError();
    give_back(object);
    return nullptr;
  }
  if (cudaGraphRetainUserObject(graph, o, 1, cudaGraphUserObjectMove) != cudaSuccess) {
    cudaGetLastError();
    cudaUserObjectRelease(o, 1);  // gives it back
    return nullptr;
  }
  return first + (kKept + lent) * kSlotWords;
}

}  // namespace

int work_slot(int dev, cudaStream_t s, uint32_t** slot) {
  if (dev < 0 || dev >= 64) return WCOMP_EUNSUPPORTED;
  *slot = nullptr;
  Work& w = g_work[dev];
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  cudaGraph_t graph = nullptr;
  unsigned long long id = 0;
  const cudaError_t e = stream_state(s, &capture, &graph, &id);
  if (e != cudaSuccess) return map_cuda(e);
  {
    std::lock_guard<std::mutex> g(g_mu);
    const int st = first_use(&w.sets, (kStreams + kKept + kLent) * kSlotWords * sizeof(uint32_t));
    if (st != WCOMP_OK) return st;
    if (capture == cudaStreamCaptureStatusNone) {
      const int number = w.streams.of(id);
      if (number >= 0) *slot = w.sets + uint64_t(number) * kSlotWords;
      return WCOMP_OK;
    }
  }
  if (capture == cudaStreamCaptureStatusActive) *slot = captured_set(dev, graph);
  return WCOMP_OK;
}

uint32_t* work_error_word(int dev) {
  if (dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> g(g_mu);
  return g_work[dev].err;
}

WCOMP_DEBUG_HOOKS(debug_hooks_q4)
}  // namespace wc

using namespace wc;

extern "C" int wcomp_q4_encode(const uint16_t* d_w, int64_t M, int64_t N, int64_t K, int group, void* stream,
                               wcomp_q4** out) {
  if (out) *out = nullptr;
  if (!d_w || !out) return WCOMP_EINVAL;
  int st = shape_ok(M, N, K, group);
  if (st != WCOMP_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  wcomp_q4* c = nullptr;
  if ((st = make_q4(M, N, K, group, s, &c)) != WCOMP_OK) return st;
  const Blocks b = blocks_of(c, 8);
  const uint32_t grid = block_grid(b);
  const bool vec = K % 8 == 0 && aligned(d_w, 16);
#define WCOMP_ENC(NG)                                                          \
  (vec ? q4_encode_kernel<NG, true><<<grid, kThreads, 0, s>>>(d_w, b)          \
       : q4_encode_kernel<NG, false><<<grid, kThreads, 0, s>>>(d_w, b))
  if (c->ng == 1) WCOMP_ENC(1);
  else if (c->ng == 2) WCOMP_ENC(2);
  else WCOMP_ENC(4);
#undef WCOMP_ENC
  count_launches(1);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    wcomp_q4_free(c, stream);
    return map_cuda(e);
  }
  *out = c;
  return WCOMP_OK;
}

extern "C" int wcomp_q4_pack(const uint8_t* d_codes, const uint16_t* d_scales, int64_t M, int64_t N, int64_t K,
                             int group, void* stream, wcomp_q4** out) {
  if (out) *out = nullptr;
  if (!d_codes || !d_scales || !out) return WCOMP_EINVAL;
  int st = shape_ok(M, N, K, group);
  if (st != WCOMP_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  wcomp_q4* c = nullptr;
  if ((st = make_q4(M, N, K, group, s, &c)) != WCOMP_OK) return st;
  const Blocks b = blocks_of(c, 1);
  const uint32_t grid = block_grid(b);
  if (c->ng == 1) q4_pack_kernel<1><<<grid, kThreads, 0, s>>>(d_codes, d_scales, b);
  else if (c->ng == 2) q4_pack_kernel<2><<<grid, kThreads, 0, s>>>(d_codes, d_scales, b);
  else q4_pack_kernel<4><<<grid, kThreads, 0, s>>>(d_codes, d_scales, b);
  count_launches(1);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    wcomp_q4_free(c, stream);
    return map_cuda(e);
  }
  *out = c;
  return WCOMP_OK;
}

extern "C" int wcomp_q4_unpack(const wcomp_q4* c, uint8_t* d_codes, uint16_t* d_scales, void* stream) {
  if (!c || !d_codes || !d_scales || !on_device(c)) return WCOMP_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Blocks b = blocks_of(c, 1);
  const uint32_t grid = block_grid(b);
  if (c->ng == 1) q4_unpack_kernel<1><<<grid, kThreads, 0, s>>>(b, d_codes, d_scales);
  else if (c->ng == 2) q4_unpack_kernel<2><<<grid, kThreads, 0, s>>>(b, d_codes, d_scales);
  else q4_unpack_kernel<4><<<grid, kThreads, 0, s>>>(b, d_codes, d_scales);
  count_launches(1);
  return map_cuda(cudaGetLastError());
}

extern "C" int wcomp_q4_decode(const wcomp_q4* c, uint16_t* d_out, void* stream) {
  if (!c || !d_out || !on_device(c)) return WCOMP_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Blocks b = blocks_of(c, 1);
  const uint32_t grid = block_grid(b);
  const bool vec = c->K % 8 == 0 && aligned(d_out, 16);
#define WCOMP_DEC(NG)                                                            \
  (vec ? q4_decode_kernel<NG, true><<<grid, kThreads, 0, s>>>(b, d_out)          \
       : q4_decode_kernel<NG, false><<<grid, kThreads, 0, s>>>(b, d_out))
  if (c->ng == 1) WCOMP_DEC(1);
  else if (c->ng == 2) WCOMP_DEC(2);
  else WCOMP_DEC(4);
#undef WCOMP_DEC
  count_launches(1);
  return map_cuda(cudaGetLastError());
}

extern "C" int wcomp_q4_gemv(const wcomp_q4* c, const uint16_t* d_x, int B, float* d_y, void* stream) {
  if (!c || !d_x || !d_y || B < 1 || B > 16 || c->M != 1 || !on_device(c)) return WCOMP_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  GemvArgs p{};
  p.w = c->d;
  p.y = d_y;
  p.N = uint64_t(c->N);
  p.cuts.steps = uint32_t(c->blocks);
  p.cuts.units = uint32_t(c->tiles);
  p.B = B;
  p.x = d_x;
  p.K = uint64_t(c->K);
  return c->ng == 1   ? dispatch_gemv<1>(p, c->device, s)
         : c->ng == 2 ? dispatch_gemv<2>(p, c->device, s)
                      : dispatch_gemv<4>(p, c->device, s);
}

extern "C" int wcomp_q4_info(const wcomp_q4* c, wcomp_q4_info_t* info) {
  if (!c || !info) return WCOMP_EINVAL;
  info->M = c->M;
  info->N = c->N;
  info->K = c->K;
  info->group = c->group;
  info->pad_ = 0;
  info->bytes = uint64_t(c->M) * c->matrix_bytes();
  return WCOMP_OK;
}

extern "C" void wcomp_q4_free(wcomp_q4* c, void* stream) {
  if (!c) return;
  if (c->d) cudaFreeAsync(c->d, static_cast<cudaStream_t>(stream));
  delete c;
}
