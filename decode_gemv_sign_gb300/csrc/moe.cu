// A whole mixture-of-experts layer for 1..16 tokens in one kernel.
//
//   l[t, e] = x[t] . R[e],   p = softmax(l[t]) or sigmoid(l[t]),
//   the k experts of largest p + bias (ties: the lowest index), weights
//   v[t, j] = factor * p_j (/ sum_j p_j),
//   y[t] = sum_j v[t, j] D_j (silu(G_j x[t]) * (U_j x[t])).
//
// For a few tokens the layer streams the chosen experts' weights once and does
// little with them, so the kernel is built around that stream: a persistent
// cooperative grid runs three phases with a grid barrier between them, and the
// barrier's wait is spent with the next phase's weights in flight where they
// are known.
//
//   A  router logits on the tensor cores, H split over warps and CTAs; each
//      part goes to the workspace in fp32.
//   -- barrier; every CTA then adds the parts in order, chooses the experts
//      and lists the (expert, token) pairs by expert, the same in every CTA.
//   B  units of 16 gate rows and the 16 matching up rows of one chosen expert
//      with all its tokens: the eight warps split H, their sums meet in shared
//      memory, and h = silu(g) u leaves as two BF16 values, high and low part
//      (16 significant bits, so h costs the result no visible rounding).
//   -- barrier; the first copies of phase C are issued before it.
//   C  units of 16 output rows: the warps split the chosen experts' k-steps,
//      all experts in a row, evenly; at an expert's end a warp adds its sums,
//      weighted, to its own [token][row] accumulators (fp32, shared memory),
//      and at the unit's end the warps' accumulators are added in order.
//
// Every sum has a fixed order: results repeat bit for bit.
#include <string.h>

#include <algorithm>
#include <atomic>

#include "tile.cuh"

namespace wc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxT = 16;
constexpr int kMaxK = 16;
constexpr int kMaxE = 1024;
constexpr int kMaxPairs = kMaxT * kMaxK;
constexpr uint64_t kBarrierNs = 1000000000ull;  // how long a CTA waits for the others (1 s)

struct Weights {
  const uint8_t* p;       // 4-bit blocks, or BF16 rows
  uint64_t expert_bytes;  // from one expert to the next
  uint32_t N, K;
};

struct MoeParams {
  const uint16_t* x;  // as the caller gave it, [T, H]
  const uint16_t* xs; // rows the products read: x, or its padded copy
  uint64_t ldx;
  uint32_t kx;
  uint16_t* xpad;     // set: phase A fills the padded copy
  const uint16_t* router;
  const float* bias;
  Weights gate, up, down;
  uint16_t* y;
  int32_t* ids;       // optional [T, k]
  float* weights;     // optional [T, k]
  float* logits;      // [splits][T][E]
  uint16_t* h;        // [pairs][2][Fp]
  uint32_t T, E, k, H, F, Fp, splits;
  int scoring, renorm;
  float factor;
  uint32_t* counters; // [0], [1] barriers, [2] CTAs done; zero
  uint32_t* err;
};

// The chosen experts, built alike in every CTA.
struct Lists {
  float w[kMaxPairs];         // pair's weight, pairs sorted by (expert, token)
  uint16_t expert[kMaxPairs]; // chosen expert a
  uint16_t start[kMaxPairs + 1];  // first pair of expert a
  uint8_t tok[kMaxPairs];     // pair's token
  uint32_t active;            // experts chosen by at least one token
};

struct Choice {  // before sorting, pair t * k + j
  float w[kMaxPairs];
  uint16_t e[kMaxPairs];
  uint8_t first[kMaxPairs];   // sorted position starts an expert
  uint16_t es[kMaxPairs];     // experts, sorted
};

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Wait until every CTA of the (cooperative, so resident) grid has arrived.
// Bounded: after kBarrierNs the error word is set and false comes back, to
// every thread of the CTA.
__device__ bool grid_barrier(uint32_t* counter, uint32_t* err, uint32_t* s_ok) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(counter, 1u);
    uint32_t v, ok = 1u;
    uint64_t deadline = 0;
    while (true) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
      if (v >= gridDim.x) break;
      const uint64_t t = now_ns();
      if (!deadline) deadline = t + kBarrierNs;
      if (t > deadline) {
        ok = 0u;
        atomicOr(err, 1u);
        break;
      }
    }
    __threadfence();
    *s_ok = ok;
  }
  __syncthreads();
  return *s_ok != 0u;
}

// Order-preserving integer of a score; NaN ranks below everything.
__device__ __forceinline__ uint32_t rank_key(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Scores and choice of token t by one warp; sc: this warp's E scores in shared
// memory.  Lane l owns experts l, l + 32, ... (at most 32 of them).
__device__ void choose(const MoeParams& p, uint32_t t, int lane, float* sc, Choice& ch) {
  float mx = -INFINITY;
  for (uint32_t e = lane; e < p.E; e += 32) {
    float l = 0.f;
    for (uint32_t s = 0; s < p.splits; ++s) l += __ldcg(p.logits + (uint64_t(s) * p.T + t) * p.E + e);
    sc[e] = l;
    mx = fmaxf(mx, l);
  }
  mx = warp_max(mx);
  if (p.scoring == WCOMP_MOE_SOFTMAX) {
    float sum = 0.f;
    for (uint32_t e = lane; e < p.E; e += 32) {
      const float v = expf(sc[e] - mx);
      sc[e] = v;
      sum += v;
    }
    sum = warp_sum(sum);
    for (uint32_t e = lane; e < p.E; e += 32) sc[e] = sc[e] / sum;
  } else {
    for (uint32_t e = lane; e < p.E; e += 32) sc[e] = 1.f / (1.f + expf(-sc[e]));
  }
  uint32_t taken = 0u;  // bit i: this lane's i-th expert is chosen
  float psum = 0.f;
  for (uint32_t j = 0; j < p.k; ++j) {
    uint64_t best = 0u;  // key, then the complement of the index: ties go to the lowest
    uint32_t i = 0;
    for (uint32_t e = lane; e < p.E; e += 32, ++i) {
      if ((taken >> i) & 1u) continue;
      const float by = p.bias ? sc[e] + p.bias[e] : sc[e];
      const uint64_t key = (uint64_t(rank_key(by)) << 32) | (0xFFFFFFFFu - e);
      best = key > best ? key : best;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const uint64_t v = __shfl_xor_sync(0xffffffffu, best, o);
      best = v > best ? v : best;
    }
    const uint32_t e = 0xFFFFFFFFu - uint32_t(best);  // E >= k: there is always one left
    if ((e & 31u) == uint32_t(lane)) taken |= 1u << (e >> 5);
    const float v = sc[e];
    psum += v;
    if (lane == 0) {
      ch.e[t * p.k + j] = uint16_t(e);
      ch.w[t * p.k + j] = v;
    }
  }
  __syncwarp();
  const float mul = p.renorm ? p.factor / (psum != psum ? psum : fmaxf(psum, 1e-20f)) : p.factor;
  if (uint32_t(lane) < p.k) ch.w[t * p.k + lane] *= mul;
}

// Pairs sorted by (expert, token), and where each chosen expert's pairs begin.
__device__ void build_lists(const MoeParams& p, Choice& ch, Lists& L) {
  const uint32_t n = p.T * p.k, i = threadIdx.x;
  uint32_t rank = 0;
  if (i < n) {
    const uint32_t key = uint32_t(ch.e[i]) * kMaxT + i / p.k;
    for (uint32_t j = 0; j < n; ++j) rank += uint32_t(ch.e[j]) * kMaxT + j / p.k < key;
    L.w[rank] = ch.w[i];
    L.tok[rank] = uint8_t(i / p.k);
    ch.es[rank] = ch.e[i];
  }
  __syncthreads();
  const bool first = i < n && (i == 0 || ch.es[i] != ch.es[i - 1]);
  if (i < n) ch.first[i] = first;
  __syncthreads();
  if (first) {
    uint32_t a = 0;
    for (uint32_t j = 0; j < i; ++j) a += ch.first[j];
    L.expert[a] = ch.es[i];
    L.start[a] = uint16_t(i);
  }
  if (i == n - 1) {
    uint32_t a = 0;
    for (uint32_t j = 0; j < n; ++j) a += ch.first[j];
    L.active = a;
    L.start[a] = uint16_t(n);
  }
  __syncthreads();
}

__device__ __forceinline__ void split_bf16(float v, uint16_t& hi, uint16_t& lo) {
  const uint32_t u = __float_as_uint(v);
  auto round = [](uint32_t b) { return (b & 0x7FFFFFFFu) > 0x7F800000u ? 0x7FC0u : (b + 0x7FFFu + ((b >> 16) & 1u)) >> 16; };
  const uint32_t h = round(u);
  hi = uint16_t(h);
  // what an infinity or NaN leaves is nothing
  lo = (h & 0x7F80u) == 0x7F80u ? uint16_t(0) : uint16_t(round(__float_as_uint(v - __uint_as_float(h << 16))));
}

template <class SRC>
__device__ __forceinline__ typename SRC::Tile expert_tile(const Weights& w, uint32_t e, uint32_t tile) {
  if constexpr (SRC::kCols == kQ4Cols) {
    const uint64_t steps = cdiv(w.K, kQ4Cols);
    return {w.p + e * w.expert_bytes + tile * steps * q4_block_bytes(SRC::NG)};
  } else {
    const uint32_t r0 = tile * kTileRows;
    return {reinterpret_cast<const uint16_t*>(w.p + e * w.expert_bytes) + uint64_t(r0) * w.K,
            w.N - r0 < kTileRows ? w.N - r0 : uint32_t(kTileRows), w.K};
  }
}

template <class SRC>
constexpr int moe_depth() { return SRC::kCols == kBfCols ? 2 : SRC::kStage > 1400 ? 3 : 4; }
template <class SRC>
constexpr uint32_t moe_ring() { return moe_depth<SRC>() * 2 * SRC::kStage; }  // one warp's
// Shared memory after the rings, used by one phase at a time: the scores
// (8 warps x 1024), B's parts (2 x 8 warps x 2 tiles x 2 x 512 bytes), C's
// accumulators (2 x 8 warps x 16 tokens x 16 rows)
constexpr uint32_t kShare = 32768;

template <class SRC, int NT, class ISSUE>
__device__ __forceinline__ void run_gate_up(const MoeParams& p, const Lists& L, uint32_t a, uint32_t ft, uint32_t w0,
                                            uint32_t w1, uint32_t ring, uint32_t& slot, int lane, int warp, float* part,
                                            ISSUE& issue) {
  constexpr int D = moe_depth<SRC>();
  const uint32_t p0 = L.start[a], n = L.start[a + 1] - p0;
  XRows<NT> x;
  x.K = p.kx;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const uint32_t c = (uint32_t(lane) >> 2) + 8 * nt;
    x.p[nt] = c < n ? p.xs + uint64_t(L.tok[p0 + c]) * p.ldx : nullptr;
  }
  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[m][nt][0] = acc[m][nt][1] = acc[m][nt][2] = acc[m][nt][3] = 0.f;
  for (uint32_t s = w0; s < w1; ++s) {
    cp_async_wait<D - 1>();
    // x (or its copy made in phase A) was written before this grid's barrier
    SRC::template step<2, NT, false>(ring + slot * 2 * SRC::kStage, s, lane, x, acc);
    issue();
    slot = slot + 1 == D ? 0 : slot + 1;
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      *reinterpret_cast<float4*>(part + ((warp * 2 + m) * 2 + nt) * 128 + lane * 4) =
          make_float4(acc[m][nt][0], acc[m][nt][1], acc[m][nt][2], acc[m][nt][3]);
  __syncthreads();
  // thread (row j, pair c): add the warps in order
  const uint32_t j = threadIdx.x % kTileRows, c = threadIdx.x / kTileRows;
  if (c < n) {
    const float* src = part + (c >> 3) * 128 + ((j & 7) * 4 + ((c & 7) >> 1)) * 4 + (j >> 3) * 2 + (c & 1);
    float g = 0.f, u = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      g += src[w * 512];
      u += src[w * 512 + 256];
    }
    const uint32_t row = ft * kTileRows + j;
    uint16_t hi = 0, lo = 0;
    if (row < p.F) split_bf16(g / (1.f + expf(-g)) * u, hi, lo);
    uint16_t* h = p.h + uint64_t(p0 + c) * 2 * p.Fp;
    h[row] = hi;
    h[p.Fp + row] = lo;
    if (ft + 1 == cdiv(p.F, kTileRows))  // zeros up to the row's padded end
      for (uint32_t f = row + kTileRows; f < p.Fp; f += kTileRows) h[f] = h[p.Fp + f] = 0;
  }
}

// One expert's share [k0, k1) of phase C for this warp, added to its
// accumulators.  Columns 2c and 2c + 1 of the MMA are the high and low part of
// pair c, so one lane holds both sums.
template <class SRC, int NT, class ISSUE>
__device__ __forceinline__ void run_down(const MoeParams& p, const Lists& L, uint32_t a, uint32_t k0, uint32_t k1,
                                         uint32_t ring, uint32_t& slot, int lane, float* ys, ISSUE& issue) {
  constexpr int D = 2 * moe_depth<SRC>();
  const uint32_t p0 = L.start[a], n = L.start[a + 1] - p0;
  XRows<NT> x;
  x.K = p.Fp;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const uint32_t c = (uint32_t(lane) >> 2) + 8 * nt;
    x.p[nt] = (c >> 1) < n ? p.h + (uint64_t(p0 + (c >> 1)) * 2 + (c & 1)) * p.Fp : nullptr;
  }
  float acc[1][NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) acc[0][nt][0] = acc[0][nt][1] = acc[0][nt][2] = acc[0][nt][3] = 0.f;
  for (uint32_t s = k0; s < k1; ++s) {
    cp_async_wait<D - 1>();
    SRC::template step<1, NT, false>(ring + slot * SRC::kStage, s, lane, x, acc);
    issue();
    slot = slot + 1 == D ? 0 : slot + 1;
  }
  const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const uint32_t c = 4 * nt + t;
    if (c < n) {
      float* y = ys + L.tok[p0 + c] * kTileRows;
      const float w = L.w[p0 + c];
      y[g] = fmaf(w, acc[0][nt][0] + acc[0][nt][1], y[g]);
      y[g + 8] = fmaf(w, acc[0][nt][2] + acc[0][nt][3], y[g + 8]);
    }
  }
  __syncwarp();  // the next expert's pairs may touch the same tokens from other lanes
}

template <class SRC, bool RVEC>
__global__ void __launch_bounds__(kThreads, 2) moe_kernel(const __grid_constant__ MoeParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Lists L;
  __shared__ Choice ch;
  __shared__ uint32_t s_ok;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t ring = smem_u32(smem) + uint32_t(warp) * moe_ring<SRC>();
  float* share = reinterpret_cast<float*>(smem + kWarps * moe_ring<SRC>());

  // ---- A: router logits
  {
    using R = BfSrc<RVEC>;
    const Weights rw{reinterpret_cast<const uint8_t*>(p.router), 0, p.E, p.H};
    const uint32_t tiles = uint32_t(cdiv(p.E, kTileRows)), steps = uint32_t(cdiv(p.H, kBfCols));
    constexpr int D = int(moe_ring<SRC>() / R::kStage);
    int par = 0;
    for (uint32_t u = blockIdx.x; u < tiles * p.splits; u += gridDim.x) {
      const uint32_t tile = u / p.splits, sp = u % p.splits;
      const uint32_t part_i = sp * kWarps + warp, parts = p.splits * kWarps;
      const uint32_t k0 = uint32_t(uint64_t(steps) * part_i / parts), k1 = uint32_t(uint64_t(steps) * (part_i + 1) / parts);
      const auto t = expert_tile<R>(rw, 0, tile);
      float acc[1][2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) acc[0][nt][0] = acc[0][nt][1] = acc[0][nt][2] = acc[0][nt][3] = 0.f;
      for (int i = 0; i < D; ++i) {
        if (k0 + i < k1) R::issue(t, k0 + i, ring + i * R::kStage, lane);
        cp_async_commit();
      }
      for (uint32_t s = k0; s < k1; ++s) {
        const uint32_t st = ring + (s - k0) % D * R::kStage;
        cp_async_wait<D - 1>();
        // activations of this k-step straight from x, whatever its alignment
        uint32_t xv[2][8];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const uint32_t b = (uint32_t(lane) >> 2) + 8 * nt, c = s * kBfCols + 16 * (uint32_t(lane) & 3);
#pragma unroll
          for (int i = 0; i < 8; ++i) xv[nt][i] = 0u;
          if (b < p.T) {
            const uint16_t* xr = p.x + uint64_t(b) * p.H;
            if (!p.xpad) {
              if (c < p.H) ld_x32<true>(xr + c, xv[nt]);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (c + e < p.H) xv[nt][e >> 1] |= uint32_t(__ldg(xr + c + e)) << (16 * (e & 1));
            }
          }
        }
        const uint32_t sm = st + lane * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 wg = lds_v4(sm + h * 512), wh = lds_v4(sm + 1024 + h * 512);
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            mma16816(acc[0][nt], wg.x, wh.x, wg.y, wh.y, xv[nt][4 * h], xv[nt][4 * h + 1]);
            mma16816(acc[0][nt], wg.z, wh.z, wg.w, wh.w, xv[nt][4 * h + 2], xv[nt][4 * h + 3]);
          }
        }
        if (s + D < k1) R::issue(t, s + D, st, lane);
        cp_async_commit();
      }
      float* part = share + par * (kWarps * 256);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
        *reinterpret_cast<float4*>(part + (warp * 2 + nt) * 128 + lane * 4) =
            make_float4(acc[0][nt][0], acc[0][nt][1], acc[0][nt][2], acc[0][nt][3]);
      __syncthreads();
      par ^= 1;
      const uint32_t j = threadIdx.x % kTileRows, b = threadIdx.x / kTileRows, e = tile * kTileRows + j;
      if (b < p.T && e < p.E) {
        const float* src = part + (b >> 3) * 128 + ((j & 7) * 4 + ((b & 7) >> 1)) * 4 + (j >> 3) * 2 + (b & 1);
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += src[w * 256];
        p.logits[(uint64_t(sp) * p.T + b) * p.E + e] = v;
      }
    }
    if (p.xpad)
      pad_rows(p.x, p.H, p.ldx, p.T, p.xpad, uint64_t(blockIdx.x) * kThreads + threadIdx.x,
               uint64_t(gridDim.x) * kThreads);
  }
  bool ok = grid_barrier(p.counters, p.err, &s_ok);
  if (ok) {
    // ---- the choice, alike in every CTA
    for (uint32_t t = warp; t < p.T; t += kWarps) choose(p, t, lane, share + warp * kMaxE, ch);
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x < p.T * p.k) {
      if (p.ids) p.ids[threadIdx.x] = ch.e[threadIdx.x];
      if (p.weights) p.weights[threadIdx.x] = ch.w[threadIdx.x];
    }
    build_lists(p, ch, L);

    // ---- B: gate and up
    {
      const uint32_t ft_n = uint32_t(cdiv(p.F, kTileRows)), units = L.active * ft_n;
      const uint32_t steps = uint32_t(cdiv(p.H, SRC::kCols));
      const uint32_t w0 = uint32_t(uint64_t(steps) * warp / kWarps), w1 = uint32_t(uint64_t(steps) * (warp + 1) / kWarps);
      constexpr int D = moe_depth<SRC>();
      uint32_t iu = w0 < w1 ? blockIdx.x : units, is = w0, islot = 0;
      typename SRC::Tile tg{}, tu{};
      auto enter = [&]() {
        if (iu >= units) return;
        const uint32_t e = L.expert[iu / ft_n], ft = iu % ft_n;
        tg = expert_tile<SRC>(p.gate, e, ft);
        tu = expert_tile<SRC>(p.up, e, ft);
      };
      auto issue = [&]() {
        if (iu < units) {
          const uint32_t st = ring + islot * 2 * SRC::kStage;
          SRC::issue(tg, is, st, lane);
          SRC::issue(tu, is, st + SRC::kStage, lane);
          if (++is == w1) {
            is = w0;
            iu += gridDim.x;
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
      for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
        const uint32_t a = u / ft_n, ft = u % ft_n;
        float* part = share + par * (kWarps * 512);
        par ^= 1;
        if (L.start[a + 1] - L.start[a] <= 8)
          run_gate_up<SRC, 1>(p, L, a, ft, w0, w1, ring, slot, lane, warp, part, issue);
        else
          run_gate_up<SRC, 2>(p, L, a, ft, w0, w1, ring, slot, lane, warp, part, issue);
      }
      cp_async_wait<0>();
    }

    // ---- C: down and the weighted sum
    {
      const uint32_t ht_n = uint32_t(cdiv(p.H, kTileRows)), steps = uint32_t(cdiv(p.F, SRC::kCols));
      const uint32_t all = L.active * steps;
      const uint32_t w0 = uint32_t(uint64_t(all) * warp / kWarps), w1 = uint32_t(uint64_t(all) * (warp + 1) / kWarps);
      constexpr int D = 2 * moe_depth<SRC>();
      uint32_t iu = w0 < w1 ? blockIdx.x : ht_n, is = w0, islot = 0, ik = 0, ia = 0;
      typename SRC::Tile td{};
      auto enter = [&]() {
        ia = is / steps;
        ik = is % steps;
        td = expert_tile<SRC>(p.down, L.expert[ia], iu);
      };
      auto issue = [&]() {
        if (iu < ht_n) {
          SRC::issue(td, ik, ring + islot * SRC::kStage, lane);
          ++ik;
          if (++is == w1) {
            is = w0;
            iu += gridDim.x;
            if (iu < ht_n) enter();
          } else if (ik == steps) {
            enter();
          }
        }
        cp_async_commit();
        islot = islot + 1 == D ? 0 : islot + 1;
      };
      if (iu < ht_n) enter();
#pragma unroll
      for (int i = 0; i < D; ++i) issue();
      ok = grid_barrier(p.counters + 1, p.err, &s_ok);
      if (ok) {
        uint32_t slot = 0;
        int par = 0;
        for (uint32_t u = blockIdx.x; u < ht_n; u += gridDim.x) {
          float* acc0 = share + par * (kWarps * kMaxT * kTileRows);
          float* ys = acc0 + warp * (kMaxT * kTileRows);
          par ^= 1;
          for (uint32_t i = lane; i < p.T * kTileRows; i += 32) ys[i] = 0.f;
          __syncwarp();
          for (uint32_t s = w0; s < w1;) {
            const uint32_t a = s / steps, k0 = s % steps;
            const uint32_t k1 = w1 - s < steps - k0 ? k0 + (w1 - s) : steps;
            const uint32_t n = L.start[a + 1] - L.start[a];
            if (n <= 4)
              run_down<SRC, 1>(p, L, a, k0, k1, ring, slot, lane, ys, issue);
            else if (n <= 8)
              run_down<SRC, 2>(p, L, a, k0, k1, ring, slot, lane, ys, issue);
            else
              run_down<SRC, 4>(p, L, a, k0, k1, ring, slot, lane, ys, issue);
            s += k1 - k0;
          }
          __syncthreads();
          const uint32_t j = threadIdx.x % kTileRows, t = threadIdx.x / kTileRows, row = u * kTileRows + j;
          if (t < p.T && row < p.H) {
            float v = 0.f;
            for (int w = 0; w < kWarps; ++w) v += acc0[(w * kMaxT + t) * kTileRows + j];
            const uint32_t b = __float_as_uint(v);
            p.y[uint64_t(t) * p.H + row] =
                (b & 0x7FFFFFFFu) > 0x7F800000u ? uint16_t(0x7FC0) : uint16_t((b + 0x7FFFu + ((b >> 16) & 1u)) >> 16);
          }
        }
      }
      cp_async_wait<0>();
    }
  }
  // the last CTA to finish leaves the counters at zero for their next launch
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(p.counters + 2, 1u) == gridDim.x - 1) {
      p.counters[0] = p.counters[1] = p.counters[2] = 0u;
      __threadfence();
    }
  }
}

template <class SRC, bool RVEC>
int launch_moe(MoeParams& p, int dev, cudaStream_t s) {
  static std::atomic<int> cache[64];
  auto kern = moe_kernel<SRC, RVEC>;
  constexpr uint32_t smem = kWarps * moe_ring<SRC>() + kShare;
  int per_sm = cache[dev].load(std::memory_order_acquire);
  if (!per_sm) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess)
      return map_cuda(cudaGetLastError());
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, smem);
    if (e != cudaSuccess) return map_cuda(e);
    if (per_sm < 1) return WCOMP_EUNSUPPORTED;
    cache[dev].store(per_sm, std::memory_order_release);
  }
  const uint32_t grid = uint32_t(per_sm * sm_count(dev));
  void* args[] = {&p};
  const cudaError_t e =
      cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kern), dim3(grid), dim3(kThreads), args, smem, s);
  count_launches(1);
  return map_cuda(e == cudaSuccess ? cudaGetLastError() : e);
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace
}  // namespace wc

using namespace wc;

extern "C" int wcomp_moe(const wcomp_moe_args* a, void* stream) {
  if (!a || !a->d_x || !a->d_router || !a->d_y) return WCOMP_EINVAL;
  if (a->T < 1 || a->T > kMaxT || a->E < 1 || a->top_k < 1 || a->top_k > a->E || a->H < 1 || a->F < 1)
    return WCOMP_EINVAL;
  if (a->scoring != WCOMP_MOE_SOFTMAX && a->scoring != WCOMP_MOE_SIGMOID) return WCOMP_EINVAL;
  if (a->E > kMaxE || a->top_k > kMaxK || a->H > (1 << 24) || a->F > (1 << 24)) return WCOMP_EUNSUPPORTED;
  const wcomp_q4* q[3] = {a->q4_gate, a->q4_up, a->q4_down};
  const uint16_t* w[3] = {a->d_gate, a->d_up, a->d_down};
  const bool q4 = q[0] || q[1] || q[2];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return map_cuda(e);
  if (dev < 0 || dev >= 64) return WCOMP_EUNSUPPORTED;
  for (int i = 0; i < 3; ++i) {
    // all three in one form
    if (q4 ? (!q[i] || w[i]) : !w[i]) return WCOMP_EINVAL;
    if (q4) {
      const int64_t N = i == 2 ? a->H : a->F, K = i == 2 ? a->F : a->H;
      if (q[i]->M != a->E || q[i]->N != N || q[i]->K != K || q[i]->ng != q[0]->ng || q[i]->device != dev)
        return WCOMP_EINVAL;
    }
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  MoeParams p;
  memset(&p, 0, sizeof(p));
  p.x = p.xs = a->d_x;
  p.ldx = uint64_t(a->H);
  p.kx = uint32_t(a->H);
  p.router = a->d_router;
  p.bias = a->d_bias;
  p.y = a->d_y;
  p.ids = a->d_ids;
  p.weights = a->d_weights;
  p.T = uint32_t(a->T);
  p.E = uint32_t(a->E);
  p.k = uint32_t(a->top_k);
  p.H = uint32_t(a->H);
  p.F = uint32_t(a->F);
  p.Fp = uint32_t(cdiv(uint64_t(a->F), kQ4Cols) * kQ4Cols);
  p.scoring = a->scoring;
  p.renorm = a->renormalize;
  p.factor = a->factor;
  Weights* out[3] = {&p.gate, &p.up, &p.down};
  for (int i = 0; i < 3; ++i) {
    Weights& t = *out[i];
    t.N = i == 2 ? p.H : p.F;
    t.K = i == 2 ? p.F : p.H;
    t.p = q4 ? q[i]->d : reinterpret_cast<const uint8_t*>(w[i]);
    t.expert_bytes = q4 ? q[i]->matrix_bytes() : uint64_t(2) * t.N * t.K;
  }
  // the router's k-steps split over CTAs too, up to four ways where E's tiles
  // are few; each part is one more term in every CTA's choice
  const uint32_t tiles = uint32_t(cdiv(p.E, kTileRows)), steps = uint32_t(cdiv(p.H, kBfCols));
  p.splits = std::max(1u, std::min({4u, uint32_t(sm_count(dev)) / tiles, steps / (2 * kWarps)}));
  const bool pad = a->H % 16 != 0 || !aligned(a->d_x, 32);
  const uint64_t Hp = cdiv(p.H, kQ4Cols) * kQ4Cols;
  auto round = [](uint64_t b) { return (b + 255) & ~uint64_t(255); };
  const uint64_t b_log = round(uint64_t(4) * p.splits * p.T * p.E), b_h = round(uint64_t(4) * p.T * p.k * p.Fp),
                 b_pad = pad ? round(2 * p.T * Hp) : 0;
  uint8_t* ws = nullptr;
  e = pool_alloc(reinterpret_cast<void**>(&ws), b_log + b_h + b_pad, s);
  if (e != cudaSuccess) return map_cuda(e);
  p.logits = reinterpret_cast<float*>(ws);
  p.h = reinterpret_cast<uint16_t*>(ws + b_log);
  if (pad) {
    p.xpad = reinterpret_cast<uint16_t*>(ws + b_log + b_h);
    p.xs = p.xpad;
    p.ldx = Hp;
    p.kx = uint32_t(Hp);
  }
  int st = work_slot(dev, &p.counters, &p.err);
  const bool rvec = p.H % 8 == 0 && aligned(a->d_router, 16);
  const bool wvec = p.H % 8 == 0 && p.F % 8 == 0 && aligned(a->d_gate, 16) && aligned(a->d_up, 16) && aligned(a->d_down, 16);
#define WCOMP_MOE(SRC) st = rvec ? launch_moe<SRC, true>(p, dev, s) : launch_moe<SRC, false>(p, dev, s)
  if (st == WCOMP_OK) {
    if (!q4) {
      if (wvec) WCOMP_MOE(BfSrc<true>);
      else WCOMP_MOE(BfSrc<false>);
    } else if (q[0]->ng == 1) {
      WCOMP_MOE(Q4Src<1>);
    } else if (q[0]->ng == 2) {
      WCOMP_MOE(Q4Src<2>);
    } else {
      WCOMP_MOE(Q4Src<4>);
    }
  }
#undef WCOMP_MOE
  cudaFreeAsync(ws, s);
  return st;
}
