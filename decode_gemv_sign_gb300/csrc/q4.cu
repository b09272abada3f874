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
// Quantise, read back, and the plain layouts.  One warp takes one block (16
// rows x 128 columns); lane (g, t) holds the 32 columns of its four runs in
// rows g and g + 8, so codes leave in the A-fragment order with no exchange,
// and a group's largest magnitude needs two shuffles in a quad.
// ---------------------------------------------------------------------------
struct Blocks {
  uint8_t* d;
  uint64_t N, K, tiles, blocks, total;  // total = M * tiles * blocks
};

// Block i of a batch of matrices: its first row and column, and the row index
// of its first row over all matrices.
struct At {
  uint64_t r0, k0, row;
};
__device__ __forceinline__ At block_at(const Blocks& b, uint64_t i) {
  const uint64_t tile = i / b.blocks;
  const uint64_t m = tile / b.tiles, t = tile % b.tiles;
  return {t * kTileRows, (i % b.blocks) * kQ4Cols, m * b.N + t * kTileRows};
}

__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b & 0x7FFF7FFFu));
  return d;
}

// The BF16 scale of a group whose largest magnitude (BF16 bits, NaN if it
// holds one) is m.  fp32 division and one rounding give the nearest BF16 to
// m / 7: m has 8 significant bits, so m / 7 is never nearer than 2^-12 to a
// midpoint of two BF16 values and the division's own rounding cannot cross it.
// A group with an infinity or a NaN gets the scale NaN.
__device__ __forceinline__ uint32_t scale_of(uint32_t m) {
  if (m >= 0x7F80u) return 0x7FC0u;
  const float s = __fdiv_rn(__uint_as_float(m << 16), 7.f);
  uint32_t u = __float_as_uint(s);
  u += 0x7FFFu + ((u >> 16) & 1u);
  return u >> 16;
}

// Code of one weight.  w / s has a quotient of 8-bit significands: it is
// either exactly halfway between integers or at least 2^-10 away from it, so
// w * (1 / s) (2^-23 relative error), rounded to a multiple of 2^-12 by the
// first constant, is on the right side of every halfway point, and exactly on
// it where w / s is; the second constant then rounds half to even.  Scales
// below 2^-100 (reciprocals near overflow, quotients above 7) divide and clamp.
constexpr float kSnap = 3072.f;        // 1.5 * 2^11: ulp 2^-12
constexpr float kRound = 12582920.f;   // 1.5 * 2^23 + 8: ulp 1, and the code's offset of 8
__device__ __forceinline__ uint32_t code_fast(float w, float rs) {
  return __float_as_uint(__fadd_rn(__fadd_rn(__fmaf_rn(w, rs, kSnap), -kSnap), kRound)) & 15u;
}
__device__ __forceinline__ uint32_t code_slow(float w, float s) {
  if (!(s > 0.f)) return 8u;  // scale 0 or NaN
  return uint32_t(int(fminf(fmaxf(rintf(__fdiv_rn(w, s)), -7.f), 7.f)) + 8);
}

// 8 columns of row r from column c as BF16 pairs; zeros outside the matrix.
template <bool VEC>
__device__ __forceinline__ void load8(const uint16_t* __restrict__ row, uint64_t c, uint64_t K, bool ok, uint32_t* v) {
  if constexpr (VEC) {
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    if (ok && c < K) q = ld_stream_v4(row + c);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = ok && c + 2 * e < K ? uint32_t(__ldg(row + c + 2 * e)) : 0u;
      const uint32_t hi = ok && c + 2 * e + 1 < K ? uint32_t(__ldg(row + c + 2 * e + 1)) : 0u;
      v[e] = lo | (hi << 16);
    }
  }
}

template <int NG, bool VEC>
__global__ void __launch_bounds__(kThreads) q4_encode_kernel(const uint16_t* __restrict__ w,
                                                             const __grid_constant__ Blocks b) {
  const int lane = threadIdx.x & 31;
  const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
  for (uint64_t i = uint64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < b.total; i += uint64_t(gridDim.x) * kWarps) {
    const At a = block_at(b, i);
    uint32_t v[2][4][4];  // row half, run, pairs
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool ok = a.r0 + g + 8 * r < b.N;
      const uint16_t* row = w + (a.row + g + 8 * r) * b.K;
#pragma unroll
      for (int q = 0; q < 4; ++q) load8<VEC>(row, a.k0 + q4_col<NG>(q, t), b.K, ok, v[r][q]);
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
        m = abs_max2(m, m >> 16) & 0xFFFFu;
        sc[r][j] = scale_of(m);
      }
    uint32_t words[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) words[j] = 0u;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float s = __uint_as_float(sc[r][q * NG / 4] << 16);
        if (s >= 0x1p-100f) {
          const float rs = __frcp_rn(s);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t p = uint32_t(r) + 2 * (e & 1);
            words[2 * q + (e >> 1)] |= (code_fast(bf16_lo(v[r][q][e]), rs) << (4 * p)) |
                                       (code_fast(bf16_hi(v[r][q][e]), rs) << (4 * p + 16));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t p = uint32_t(r) + 2 * (e & 1);
            words[2 * q + (e >> 1)] |= (code_slow(bf16_lo(v[r][q][e]), s) << (4 * p)) |
                                       (code_slow(bf16_hi(v[r][q][e]), s) << (4 * p + 16));
          }
        }
      }
    uint8_t* out = b.d + i * q4_block_bytes(NG);
    *reinterpret_cast<uint4*>(out + lane * 16) = make_uint4(words[0], words[1], words[2], words[3]);
    *reinterpret_cast<uint4*>(out + 512 + lane * 16) = make_uint4(words[4], words[5], words[6], words[7]);
    if (int(t) < NG) {  // lane t of a quad writes group t's scales
      uint32_t s2 = sc[0][0] | (sc[1][0] << 16);
#pragma unroll
      for (int j = 1; j < NG; ++j)
        if (int(t) == j) s2 = sc[0][j] | (sc[1][j] << 16);
      *reinterpret_cast<uint32_t*>(out + 1024 + (g * NG + t) * 4) = s2;
    }
  }
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// (c - 8) * s is an integer of at most 4 bits times an 8-bit significand: the
// BF16 multiply rounds the exact product once.
template <int NG, bool VEC>
__global__ void __launch_bounds__(kThreads) q4_decode_kernel(const __grid_constant__ Blocks b,
                                                             uint16_t* __restrict__ out) {
  const int lane = threadIdx.x & 31;
  const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
  for (uint64_t i = uint64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < b.total; i += uint64_t(gridDim.x) * kWarps) {
    const At a = block_at(b, i);
    const uint8_t* in = b.d + i * q4_block_bytes(NG);
    const uint4 c0 = ld_stream_v4(in + lane * 16), c1 = ld_stream_v4(in + 512 + lane * 16);
    const uint32_t cw[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    uint32_t sc[NG];
#pragma unroll
    for (int j = 0; j < NG; ++j) sc[j] = ld_stream_u32(in + 1024 + (g * NG + j) * 4);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (a.r0 + g + 8 * r >= b.N) continue;
      uint16_t* row = out + (a.row + g + 8 * r) * b.K;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t s2 = prmt(sc[q * NG / 4], 0u, r ? 0x3232u : 0x1010u);
        uint32_t v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = mul2(q4_pair(cw[2 * q + (e >> 1)], r + 2 * (e & 1)), s2);
        const uint64_t c = a.k0 + q4_col<NG>(q, t);
        if constexpr (VEC) {
          if (c < b.K) *reinterpret_cast<uint4*>(row + c) = make_uint4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < b.K) row[c + e] = uint16_t(v[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
  }
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
  const uint64_t pitch = (b.K + 1) / 2, groups = cdiv(b.K, kQ4Cols / NG);
  for (uint64_t i = uint64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < b.total; i += uint64_t(gridDim.x) * kWarps) {
    const At a = block_at(b, i);
    uint32_t words[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) words[j] = 0u;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool ok = a.r0 + g + 8 * r < b.N;
      const uint8_t* row = codes + (a.row + g + 8 * r) * pitch;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint64_t c = a.k0 + q4_col<NG>(q, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t lo = 8u, hi = 8u;
          if (ok && c + 2 * e < b.K) {
            const uint32_t byte = row[(c >> 1) + e];
            lo = byte & 15u;
            if (c + 2 * e + 1 < b.K) hi = byte >> 4;
          }
          const uint32_t p = uint32_t(r) + 2 * (e & 1);
          words[2 * q + (e >> 1)] |= (lo << (4 * p)) | (hi << (4 * p + 16));
        }
      }
    }
    uint8_t* out = b.d + i * q4_block_bytes(NG);
    *reinterpret_cast<uint4*>(out + lane * 16) = make_uint4(words[0], words[1], words[2], words[3]);
    *reinterpret_cast<uint4*>(out + 512 + lane * 16) = make_uint4(words[4], words[5], words[6], words[7]);
    if (int(t) < NG) {
      const uint64_t j = a.k0 / (kQ4Cols / NG) + t;
      uint32_t s2 = 0u;
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (a.r0 + g + 8 * r < b.N && j < groups)
          s2 |= uint32_t(scales[(a.row + g + 8 * r) * groups + j]) << (16 * r);
      *reinterpret_cast<uint32_t*>(out + 1024 + (g * NG + t) * 4) = s2;
    }
  }
}

template <int NG>
__global__ void __launch_bounds__(kThreads) q4_unpack_kernel(const __grid_constant__ Blocks b,
                                                             uint8_t* __restrict__ codes,
                                                             uint16_t* __restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
  const uint64_t pitch = (b.K + 1) / 2, groups = cdiv(b.K, kQ4Cols / NG);
  for (uint64_t i = uint64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < b.total; i += uint64_t(gridDim.x) * kWarps) {
    const At a = block_at(b, i);
    const uint8_t* in = b.d + i * q4_block_bytes(NG);
    const uint4 c0 = ld_stream_v4(in + lane * 16), c1 = ld_stream_v4(in + 512 + lane * 16);
    const uint32_t cw[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (a.r0 + g + 8 * r >= b.N) continue;
      uint8_t* row = codes + (a.row + g + 8 * r) * pitch;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint64_t c = a.k0 + q4_col<NG>(q, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t p = uint32_t(r) + 2 * (e & 1), wv = cw[2 * q + (e >> 1)];
          if (c + 2 * e < b.K) row[(c >> 1) + e] = uint8_t(((wv >> (4 * p)) & 15u) | (((wv >> (4 * p + 16)) & 15u) << 4));
        }
      }
      const uint64_t j = a.k0 / (kQ4Cols / NG) + t;
      if (int(t) < NG && j < groups)
        scales[(a.row + g + 8 * r) * groups + j] =
            uint16_t(ld_stream_u32(in + 1024 + (g * NG + t) * 4) >> (16 * r));
    }
  }
}

// ---------------------------------------------------------------------------
// GEMV.  A CTA of 8 warps works on groups of WM x MT tiles; WK = 8 / WM warps
// share a tile's k-steps.  The launch's k-steps, row group after row group,
// are cut into one contiguous range per CTA: `split` cuts anywhere, otherwise
// ranges end on whole row groups.  A row group that lies in one CTA goes
// straight to y; of a cut one each CTA leaves its fp32 part in the workspace
// and the CTA that arrives last adds them in the order of the CTAs, so the
// result does not depend on which CTA that is.
// ---------------------------------------------------------------------------
struct GemvArgs {
  const uint8_t* w;
  const uint16_t* x;
  uint64_t ldx;         // columns per row of x
  uint32_t kx;          // readable columns of a row of x, a multiple of 16
  float* y;
  float* part;          // [2 * grid][B][rows of a group]
  uint32_t* counters;   // one per row group, zero
  uint64_t N;
  uint32_t steps;       // k-steps (blocks) of a tile
  uint32_t tiles, groups;
  int B, wm, split;
};

__host__ __device__ inline uint64_t range_start(const GemvArgs& p, uint32_t cta, uint32_t grid) {
  if (p.split) return uint64_t(p.groups) * p.steps * cta / grid;
  return uint64_t(p.groups) * cta / grid * p.steps;
}

constexpr int q4_depth(int ng, int mt) { return mt == 1 ? 6 : ng == 4 ? 3 : 4; }

template <int NG, int MT>
constexpr uint32_t q4_ring() { return kWarps * q4_depth(NG, MT) * MT * Q4Src<NG>::kStage; }

template <int NG, int MT, int NT>
__global__ void __launch_bounds__(kThreads, 2) q4_gemv_kernel(const __grid_constant__ GemvArgs p) {
  using S = Q4Src<NG>;
  constexpr int D = q4_depth(NG, MT);
  extern __shared__ __align__(16) uint8_t smem[];
  float* part = reinterpret_cast<float*>(smem + q4_ring<NG, MT>());  // [2][warp][MT][NT][lane][4]
  __shared__ uint32_t s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wk_n = kWarps / p.wm, wm = warp / wk_n, wk = warp % wk_n;
  const uint32_t ring = smem_u32(smem) + uint32_t(warp) * D * MT * S::kStage;
  const uint64_t begin = range_start(p, blockIdx.x, gridDim.x), end = range_start(p, blockIdx.x + 1, gridDim.x);
  XRows<NT> x;
  x.K = p.kx;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int b = (lane >> 2) + 8 * nt;
    x.p[nt] = b < p.B ? p.x + uint64_t(b) * p.ldx : nullptr;
  }
  const uint64_t tile_bytes = uint64_t(p.steps) * q4_block_bytes(NG);
  // A row group's part of [begin, end), and this warp's k-steps of it.
  struct Seg {
    uint32_t rg, k0, k1, w0, w1;
  };
  auto seg_at = [&](uint64_t at) {
    Seg s;
    s.rg = uint32_t(at / p.steps);
    s.k0 = uint32_t(at % p.steps);
    const uint64_t left = end - at;
    s.k1 = uint32_t(left < p.steps - s.k0 ? s.k0 + left : p.steps);
    const uint32_t len = s.k1 - s.k0;
    s.w0 = s.k0 + len * wk / wk_n;
    s.w1 = s.k0 + len * (wk + 1) / wk_n;
    if ((s.rg * p.wm + wm) * MT >= p.tiles) s.w1 = s.w0;  // no tile here
    return s;
  };
  auto tile_of = [&](const Seg& s, int m) {  // past the last tile: the last one again, its sums unused
    const uint32_t i = (s.rg * p.wm + wm) * MT + m;
    return typename S::Tile{p.w + uint64_t(i < p.tiles ? i : p.tiles - 1) * tile_bytes};
  };
  // The copy cursor runs D k-steps ahead of the sums, across row groups.
  uint64_t iat = begin;
  Seg is{};
  typename S::Tile it[MT];
  uint32_t ik = 0, islot = 0;
  auto enter = [&]() {
    while (iat < end) {
      is = seg_at(iat);
      ik = is.w0;
      if (is.w0 < is.w1) break;
      iat += is.k1 - is.k0;
    }
    if (iat < end)
#pragma unroll
      for (int m = 0; m < MT; ++m) it[m] = tile_of(is, m);
  };
  auto issue = [&]() {
    if (iat < end) {
#pragma unroll
      for (int m = 0; m < MT; ++m) S::issue(it[m], ik, ring + (islot * MT + m) * S::kStage, lane);
      if (++ik == is.w1) {
        iat += is.k1 - is.k0;
        enter();
      }
    }
    cp_async_commit();
    islot = islot + 1 == D ? 0 : islot + 1;
  };
  enter();
#pragma unroll
  for (int i = 0; i < D; ++i) issue();
  uint32_t slot = 0;
  int par = 0;
  const uint32_t rows_g = uint32_t(p.wm) * MT * kTileRows;
  for (uint64_t at = begin; at < end;) {
    const Seg s = seg_at(at);
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[m][nt][0] = acc[m][nt][1] = acc[m][nt][2] = acc[m][nt][3] = 0.f;
    for (uint32_t k = s.w0; k < s.w1; ++k) {
      cp_async_wait<D - 1>();
      S::template step<MT, NT, true>(ring + slot * MT * S::kStage, k, lane, x, acc);
      issue();
      slot = slot + 1 == D ? 0 : slot + 1;
    }
    // sum the warps of a tile in order; parts alternate by parity, so one
    // barrier per row group suffices
    float* pp = part + par * (kWarps * MT * NT * 128);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        *reinterpret_cast<float4*>(pp + ((warp * MT + m) * NT + nt) * 128 + lane * 4) =
            make_float4(acc[m][nt][0], acc[m][nt][1], acc[m][nt][2], acc[m][nt][3]);
    __syncthreads();
    par ^= 1;
    const bool whole = s.k0 == 0 && s.k1 == p.steps;
    const uint64_t row0 = uint64_t(s.rg) * rows_g;
    float* ws = whole ? nullptr : p.part + (2 * uint64_t(blockIdx.x) + (at != begin)) * p.B * rows_g;
    for (uint32_t o = threadIdx.x; o < rows_g * p.B; o += kThreads) {
      const uint32_t r = o % rows_g, b = o / rows_g;
      const uint32_t m = (r / kTileRows) % MT, wmi = r / (kTileRows * MT), j = r % kTileRows;
      const float* src = pp + ((wmi * wk_n * MT + m) * NT + (b >> 3)) * 128 + ((j & 7) * 4 + ((b & 7) >> 1)) * 4 +
                         (j >> 3) * 2 + (b & 1);
      float v = 0.f;
      for (int w = 0; w < wk_n; ++w) v += src[w * MT * NT * 128];
      if (!whole)
        ws[o] = v;
      else if (row0 + r < p.N)
        p.y[uint64_t(b) * p.N + row0 + r] = v;
    }
    if (!whole) {
      // CTAs with a share of this row group: first .. last
      const uint64_t g0 = uint64_t(s.rg) * p.steps, g1 = g0 + p.steps;
      uint32_t first = blockIdx.x, last = blockIdx.x;
      while (first > 0 && range_start(p, first, gridDim.x) > g0) --first;
      while (last + 1 < gridDim.x && range_start(p, last + 1, gridDim.x) < g1) ++last;
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        s_last = atomicAdd(p.counters + s.rg, 1u) == last - first;
        __threadfence();
      }
      __syncthreads();
      if (s_last) {
        for (uint32_t o = threadIdx.x; o < rows_g * p.B; o += kThreads) {
          const uint32_t r = o % rows_g, b = o / rows_g;
          float v = 0.f;
          for (uint32_t c = first; c <= last; ++c) {
            // a CTA's part of this row group is its first unless its range began earlier
            const uint32_t which = range_start(p, c, gridDim.x) < g0 ? 1u : 0u;
            v += __ldcg(p.part + (2 * uint64_t(c) + which) * p.B * rows_g + o);
          }
          if (row0 + r < p.N) p.y[uint64_t(b) * p.N + row0 + r] = v;
        }
        if (threadIdx.x == 0) p.counters[s.rg] = 0u;
      }
    }
    at += s.k1 - s.k0;
  }
  cp_async_wait<0>();
}

__global__ void __launch_bounds__(256) pad_rows_kernel(const uint16_t* __restrict__ x, uint64_t K, uint64_t Kp,
                                                       uint32_t B, uint16_t* __restrict__ out) {
  pad_rows(x, K, Kp, B, out, uint64_t(blockIdx.x) * 256 + threadIdx.x, uint64_t(gridDim.x) * 256);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
constexpr uint32_t kSlots = 256;
std::mutex g_mu;
uint32_t* g_work[64] = {nullptr};  // kSlots x kSlotWords counters, then the error word
std::atomic<uint32_t> g_rr{0};

template <int NG, int MT, int NT>
int prepare_gemv(int dev) {
  static std::atomic<int> cache[64];
  const uint32_t smem = q4_ring<NG, MT>() + 2 * kWarps * MT * NT * 512;
  int per_sm = cache[dev].load(std::memory_order_acquire);
  if (!per_sm) {
    auto kern = q4_gemv_kernel<NG, MT, NT>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess) return -1;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, smem) != cudaSuccess || per_sm < 1)
      return -1;
    cache[dev].store(per_sm, std::memory_order_release);
  }
  return per_sm;
}

template <int NG, int MT, int NT>
int launch_gemv(GemvArgs& p, int dev, cudaStream_t s) {
  const int per_sm = prepare_gemv<NG, MT, NT>(dev);
  if (per_sm < 0) return map_cuda(cudaGetLastError());
  const uint32_t smem = q4_ring<NG, MT>() + 2 * kWarps * MT * NT * 512;
  const uint32_t rows_g = uint32_t(p.wm) * MT * kTileRows;
  p.groups = uint32_t(cdiv(p.tiles, uint64_t(p.wm) * MT));
  uint32_t grid = uint32_t(per_sm * sm_count(dev));
  if (p.split && p.groups > kSlotWords) p.split = 0;
  const uint64_t units = p.split ? uint64_t(p.groups) * p.steps : p.groups;
  if (units < grid) grid = uint32_t(units);
  if (p.split) {
    uint32_t* err = nullptr;
    const int st = work_slot(dev, &p.counters, &err);
    if (st != WCOMP_OK) return st;
    const cudaError_t e =
        pool_alloc(reinterpret_cast<void**>(&p.part), uint64_t(2) * grid * p.B * rows_g * sizeof(float), s);
    if (e != cudaSuccess) return map_cuda(e);
  }
  q4_gemv_kernel<NG, MT, NT><<<grid, kThreads, smem, s>>>(p);
  count_launches(1);
  const cudaError_t e = cudaGetLastError();
  if (p.part) cudaFreeAsync(p.part, s);
  return map_cuda(e);
}

template <int NG>
int dispatch_gemv(GemvArgs& p, int dev, cudaStream_t s) {
  if (p.B <= 8) {
    p.wm = 1;
    p.split = 0;
    return launch_gemv<NG, 1, 1>(p, dev, s);
  }
  p.wm = 4;
  p.split = 1;
  return launch_gemv<NG, 2, 2>(p, dev, s);
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
  c->ng = kQ4Cols / group;
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

Blocks blocks_of(const wcomp_q4* c) {
  return {c->d, uint64_t(c->N), uint64_t(c->K), c->tiles, c->blocks, uint64_t(c->M) * c->tiles * c->blocks};
}

uint32_t block_grid(const Blocks& b, int dev) {
  return uint32_t(std::min<uint64_t>(cdiv(b.total, kWarps), uint64_t(sm_count(dev)) * 64));
}

bool on_device(const wcomp_q4* c) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == c->device;
}

}  // namespace

int work_slot(int dev, uint32_t** slot, uint32_t** err) {
  if (dev < 0 || dev >= 64) return WCOMP_EUNSUPPORTED;
  std::lock_guard<std::mutex> g(g_mu);
  if (!g_work[dev]) {
    uint32_t* p = nullptr;
    const size_t bytes = (kSlots * kSlotWords + 32) * sizeof(uint32_t);
    cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&p), bytes);
    if (e == cudaSuccess) e = cudaMemset(p, 0, bytes);
    if (e != cudaSuccess) {
      if (p) cudaFree(p);
      return map_cuda(e);
    }
    g_work[dev] = p;
  }
  *slot = g_work[dev] + uint64_t(g_rr.fetch_add(1, std::memory_order_relaxed) % kSlots) * kSlotWords;
  *err = g_work[dev] + kSlots * kSlotWords;
  return WCOMP_OK;
}

uint32_t* work_error_word(int dev) {
  if (dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> g(g_mu);
  return g_work[dev] ? g_work[dev] + kSlots * kSlotWords : nullptr;
}

cudaError_t work_reset(int dev, cudaStream_t s) {
  uint32_t* e = work_error_word(dev);
  if (!e) return cudaSuccess;
  return cudaMemsetAsync(e - kSlots * kSlotWords, 0, (kSlots * kSlotWords + 32) * sizeof(uint32_t), s);
}

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
  const Blocks b = blocks_of(c);
  const uint32_t grid = block_grid(b, c->device);
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
  const Blocks b = blocks_of(c);
  const uint32_t grid = block_grid(b, c->device);
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
  const Blocks b = blocks_of(c);
  const uint32_t grid = block_grid(b, c->device);
  if (c->ng == 1) q4_unpack_kernel<1><<<grid, kThreads, 0, s>>>(b, d_codes, d_scales);
  else if (c->ng == 2) q4_unpack_kernel<2><<<grid, kThreads, 0, s>>>(b, d_codes, d_scales);
  else q4_unpack_kernel<4><<<grid, kThreads, 0, s>>>(b, d_codes, d_scales);
  count_launches(1);
  return map_cuda(cudaGetLastError());
}

extern "C" int wcomp_q4_decode(const wcomp_q4* c, uint16_t* d_out, void* stream) {
  if (!c || !d_out || !on_device(c)) return WCOMP_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Blocks b = blocks_of(c);
  const uint32_t grid = block_grid(b, c->device);
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
  GemvArgs p;
  memset(&p, 0, sizeof(p));
  p.w = c->d;
  p.x = d_x;
  p.ldx = uint64_t(c->K);
  p.kx = uint32_t(c->K);
  p.y = d_y;
  p.N = uint64_t(c->N);
  p.steps = uint32_t(c->blocks);
  p.tiles = uint32_t(c->tiles);
  p.B = B;
  uint16_t* pad = nullptr;
  if (c->K % 16 != 0 || !aligned(d_x, 32)) {
    const uint64_t Kp = c->blocks * kQ4Cols;
    const cudaError_t e = pool_alloc(reinterpret_cast<void**>(&pad), uint64_t(B) * Kp * 2, s);
    if (e != cudaSuccess) return map_cuda(e);
    const uint32_t grid = uint32_t(std::min<uint64_t>(cdiv(uint64_t(B) * Kp, 256), uint64_t(sm_count(c->device)) * 4));
    pad_rows_kernel<<<grid, 256, 0, s>>>(d_x, uint64_t(c->K), Kp, uint32_t(B), pad);
    count_launches(1);
    p.x = pad;
    p.ldx = Kp;
    p.kx = uint32_t(Kp);
  }
  const int st = c->ng == 1 ? dispatch_gemv<1>(p, c->device, s)
                 : c->ng == 2 ? dispatch_gemv<2>(p, c->device, s) : dispatch_gemv<4>(p, c->device, s);
  if (pad) cudaFreeAsync(pad, s);
  return st;
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
