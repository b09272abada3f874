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
// second barrier's wait is spent with the next phase's weights in flight.
//
//   A  router logits on the tensor cores, H split over warps and CTAs; each
//      part goes to the workspace in fp32.  For 4-bit experts x becomes fp16
//      records here (tile.cuh).
//   -- barrier; every CTA then adds the parts in order, chooses the experts
//      and lists the (expert, token) pairs by expert, the same in every CTA.
//   B  units of 32 gate rows and the 32 matching up rows of one chosen expert
//      with all its tokens: the eight warps split H, their sums meet in shared
//      memory, and h = silu(g) u goes to the workspace, each pair's 32 values
//      as fp16 under their own power of two (4-bit experts: 11 significant
//      bits, an eighth of a BF16 step) or as two BF16 parts (BF16 experts: 16
//      significant bits), so h costs the BF16 result no visible rounding.
//   -- barrier.
//   C  units of 32 output rows: the k-steps of all chosen experts, one expert
//      after the other, split evenly over the warps; at an expert's end a warp
//      adds its sums, weighted, to its own [token][row] accumulators (fp32,
//      shared memory), and at the unit's end the warps' accumulators are added
//      in order.
//
// Units of B and C are cut over the CTAs, where that pays for the joins, so that
// each streams the same bytes (Cuts, tile.cuh).  Every sum has a fixed order:
// results repeat bit for bit.
//
// Measured, us (in brackets the chosen weights' bytes at a plain copy's rate):
// 8 of 128 experts of 6144 x 2048: one token BF16 108 (89), 4-bit with groups of
// 128 50 (23), 16 tokens 4-bit with groups of 32 339 (258 for the experts chosen on
// average, about 280 for these); 2 of 8 of 4096 x 11008, 16 tokens, BF16 347-360
// (316); 2 of 8 of 1024 x 512, one token 13.6 (0.9).
// Large layers are bound by the stream.  Small ones by the chain of phases: of
// one token's 50 us with 4-bit experts, 3.5 are the router, 1.5 each barrier,
// 2.4 the choice and the lists, 4 the first copies of B and C, and 6 the last
// CTAs of B, of which some have two units and some one.
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
constexpr uint32_t kSplits = 4;    // parts of a router logit (CTAs that share its H)
constexpr uint32_t kMaxGrid = (kSlotWords - 8) / 2;
constexpr uint32_t kPartFloats = 1024;  // of a unit: B 2 x 32 rows x 16 pairs, C 32 rows x 16 tokens
constexpr uint64_t kBarrierNs = 1000000000ull;  // how long a CTA waits for the others (1 s)

struct Weights {
  const uint8_t* p;       // 4-bit blocks, or BF16 rows
  uint64_t expert_bytes;  // 4-bit: from one expert to the next
  uint32_t N, K;
};

struct MoeParams {
  const uint16_t* x;      // [T, H]
  const uint8_t* xs;      // what the products read: x or its padded copy (BF16 rows), or records
  float* xf;              // records' factors
  uint64_t xs_bytes;      // from one token to the next
  uint8_t* make;          // set: phase A makes xs here
  const uint16_t* router;
  const float* bias;
  Weights w[3];           // gate, up, down
  uint16_t* y;
  int32_t* ids;           // optional [T, k]
  float* weights;         // optional [T, k]
  float* logits;          // [T][E][kSplits], parts of a logit
  float* part;            // joins: 2 x kPartFloats per CTA, once for B and once for C
  uint8_t* h;             // 4-bit: [pairs][Fp / 128] records; BF16: [pairs][2][Fp] values
  float* hf;              // 4-bit: factors [Fp / 32][256]
  uint32_t T, E, k, H, F, Fp;
  int scoring, renorm, x_vec;
  float factor;
  uint32_t* counters;     // [0], [1] barriers, [2] CTAs done, and in its upper half those whose barrier ran out; from [8]
                          // one per CTA for each of B's and C's joins; zero before and after
  uint32_t* err;
};
struct MoeMaps {
  CUtensorMap m[3];       // BF16 experts' tensor maps: gate, up, down
};

// The chosen experts, built alike in every CTA.
struct Lists {
  float w[kMaxPairs];         // pair's weight, pairs sorted by (expert, token)
  uint16_t expert[kMaxPairs]; // chosen expert a
  uint16_t start[kMaxPairs + 1];  // first pair of expert a
  uint8_t tok[kMaxPairs];     // pair's token
  uint32_t active;            // experts chosen by at least one token
};

struct Choice {  // pairs t * k + j as chosen
  float w[kMaxPairs];
  uint16_t e[kMaxPairs];
  alignas(16) uint16_t key[kMaxPairs];  // expert * 16 + token
  uint16_t sorted[kMaxPairs];           // the experts, sorted
  uint32_t firsts[kWarps];              // which sorted pairs begin an expert
};

// Wait until every CTA of the (cooperative, so resident) grid has arrived.
// Bounded: after kBarrierNs the error word is set and false comes back, to
// every thread of the CTA.
__device__ bool grid_barrier(uint32_t* counter, uint32_t* err, uint32_t* s_ok, [[maybe_unused]] bool first) {
  __syncthreads();
  if (threadIdx.x == 0) {
#if WCOMP_DEBUG
    if ((g_debug_hooks & 2u) && first && blockIdx.x == 0)  // come when the others have given up
      for (const uint64_t t = timer_ns() + kBarrierNs + kBarrierNs / 2; timer_ns() < t;) {}
#endif
    __threadfence();
    atomicAdd(counter, 1u);
    uint32_t v, ok = 1u;
    uint64_t deadline = 0;
    while (true) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
      if (v >= gridDim.x) break;
      const uint64_t t = timer_ns();
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

// Order-preserving integer of a score, above 1; NaN ranks below everything.
__device__ __forceinline__ uint32_t rank_key(float v) {
  if (v != v) return 1u;
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

// Scores and choice of token t by one warp.  Lane l owns experts l, l + 32, ...
// A round of the choice is two warp reductions: the largest key, then the
// lowest index that has it.  Up to 32 U experts stay in registers, which keeps
// their loads in flight together and a round free of searches.
__device__ __forceinline__ float logit_of(const MoeParams& p, uint32_t t, uint32_t e) {
  const float4 v = __ldcg(reinterpret_cast<const float4*>(p.logits) + t * p.E + e);
  return (v.x + v.y) + (v.z + v.w);
}
__device__ __forceinline__ void put_choice(const MoeParams& p, uint32_t t, uint32_t j, uint32_t e, float score,
                                           Choice& ch) {
  const uint32_t i = t * p.k + j;
  ch.e[i] = uint16_t(e);
  ch.key[i] = uint16_t(e * kMaxT + t);
  ch.w[i] = score;
}
// exp of a logit under the row's largest (softmax), or of its negated magnitude
// (sigmoid), and the score that follows from it.  Neither overflows, so sigmoid's
// scores keep their order down to logits of -103, where fp32 ends (1 / (1 +
// exp(-l)) would be 0 from -87 on, and a choice among such experts fall to their
// index), and the divisor is 1 to 1024, where the approximate division is right
// to two units in the last place (the exact one: 0.6 us of a small layer's 14).
__device__ __forceinline__ float score_exp(bool soft, float l, float mx) { return expf(soft ? l - mx : -fabsf(l)); }
__device__ __forceinline__ float score_of(bool soft, float l, float ex, float sum) {
  return __fdividef(soft || l < 0.f ? ex : 1.f, soft ? sum : 1.f + ex);
}
template <int U>
__device__ __forceinline__ void choose(const MoeParams& p, uint32_t t, int lane, Choice& ch) {
  const bool soft = p.scoring == WCOMP_MOE_SOFTMAX;
  float sc[U], ex[U];
  uint32_t key[U];
  float mx = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t e = lane + 32 * i;
    sc[i] = e < p.E ? logit_of(p, t, e) : -INFINITY;
    mx = fmaxf(mx, sc[i]);
  }
  mx = soft ? warp_max(mx) : 0.f;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    ex[i] = score_exp(soft, sc[i], mx);
    sum += lane + 32 * i < p.E ? ex[i] : 0.f;
  }
  sum = warp_sum(sum);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t e = lane + 32 * i;
    sc[i] = score_of(soft, sc[i], ex[i], sum);
    key[i] = e < p.E ? rank_key(p.bias ? sc[i] + p.bias[e] : sc[i]) : 0u;
  }
#pragma unroll 1
  for (uint32_t j = 0; j < p.k; ++j) {
    uint32_t best = key[0], at = 0;
#pragma unroll
    for (int i = 1; i < U; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const uint32_t e = __reduce_min_sync(0xffffffffu, best == top ? lane + 32 * at : 0xFFFFFFFFu);
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (e == uint32_t(lane) + 32 * i) {  // E >= k: one is left
        put_choice(p, t, j, e, sc[i], ch);
        key[i] = 0u;
      }
  }
}
// Any E: scores and keys in shared memory (sc: kMaxE scores, then kMaxE keys).
__device__ __forceinline__ void choose_many(const MoeParams& p, uint32_t t, int lane, float* sc, Choice& ch) {
  const bool soft = p.scoring == WCOMP_MOE_SOFTMAX;
  uint32_t* keys = reinterpret_cast<uint32_t*>(sc + kMaxE);
  float mx = -INFINITY, sum = 0.f;
#pragma unroll 4
  for (uint32_t e = lane; e < p.E; e += 32) {
    const float l = logit_of(p, t, e);
    sc[e] = l;
    mx = fmaxf(mx, l);
  }
  mx = soft ? warp_max(mx) : 0.f;
  if (soft)
    for (uint32_t e = lane; e < p.E; e += 32) sum += score_exp(true, sc[e], mx);
  sum = warp_sum(sum);
  uint32_t key = 0u, at = 0xFFFFFFFFu;
  for (uint32_t e = lane; e < p.E; e += 32) {
    const float v = score_of(soft, sc[e], score_exp(soft, sc[e], mx), sum);
    const uint32_t kk = rank_key(p.bias ? v + p.bias[e] : v);
    sc[e] = v;
    keys[e] = kk;
    if (kk > key) {
      key = kk;
      at = e;
    }
  }
  for (uint32_t j = 0; j < p.k; ++j) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, key);
    const uint32_t e = __reduce_min_sync(0xffffffffu, key == top ? at : 0xFFFFFFFFu);
    if (e == at) {
      put_choice(p, t, j, e, sc[e], ch);
      keys[e] = key = 0u;
      at = 0xFFFFFFFFu;
      for (uint32_t q = lane; q < p.E; q += 32)
        if (keys[q] > key) {
          key = keys[q];
          at = q;
        }
    }
  }
}
// The chosen scores of token t become weights.
__device__ __forceinline__ void weigh(const MoeParams& p, uint32_t t, int lane, Choice& ch) {
  __syncwarp();
  float v = uint32_t(lane) < p.k ? ch.w[t * p.k + lane] : 0.f, sum = 0.f;
  for (uint32_t j = 0; j < p.k; ++j) sum += __shfl_sync(0xffffffffu, v, j);  // in the order of the choice
  v *= p.renorm ? p.factor / (sum != sum ? sum : fmaxf(sum, 1e-20f)) : p.factor;
  if (uint32_t(lane) < p.k) ch.w[t * p.k + lane] = v;
}

// Pairs sorted by (expert, token), and where each chosen expert's pairs begin.
__device__ __forceinline__ void build_lists(const MoeParams& p, Choice& ch, Lists& L) {
  const uint32_t n = p.T * p.k, i = threadIdx.x;
  if (i >= n) ch.key[i] = 0xFFFFu;  // past every key
  __syncthreads();
  if (i < n) {
    const uint32_t key = ch.key[i];
    uint32_t rank = 0;
#pragma unroll 1
    for (uint32_t j = 0; j < n; j += 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(&ch.key[j]);
      const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) rank += uint32_t((q[c] & 0xFFFFu) < key) + uint32_t((q[c] >> 16) < key);
    }
    L.w[rank] = ch.w[i];
    L.tok[rank] = uint8_t(key % kMaxT);
    ch.sorted[rank] = uint16_t(key / kMaxT);
  }
  __syncthreads();
  const bool first = i < n && (i == 0 || ch.sorted[i] != ch.sorted[i - 1]);
  const uint32_t mask = __ballot_sync(0xffffffffu, first);
  if (i % 32 == 0) ch.firsts[i / 32] = mask;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (uint32_t w = 0; w < kWarps; ++w) {
    const uint32_t c = __popc(ch.firsts[w]);
    if (w < i / 32) before += c;
    all += c;
  }
  if (first) {
    const uint32_t a = before + __popc(mask & ((1u << (i % 32)) - 1u));
    L.expert[a] = ch.sorted[i];
    L.start[a] = uint16_t(i);
  }
  if (i == 0) {
    L.active = all;
    L.start[all] = uint16_t(n);
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

// Matrix i (gate, up, down) of expert e at k-step `step` of 32-row tile `tile`.
template <class SRC>
__device__ __forceinline__ typename SRC::Cursor expert_at(const MoeParams& p, const MoeMaps& maps, int i, uint32_t e,
                                                          uint32_t tile, uint32_t step) {
  const Weights& w = p.w[i];
  if constexpr (SRC::NG > 0) {
    return SRC::at(w.p + e * w.expert_bytes, uint32_t(cdiv(w.K, kQ4Cols)), tile, step);
  } else {
    return SRC::at(&maps.m[i], reinterpret_cast<const uint16_t*>(w.p), uint64_t(p.E) * w.N,
                   uint64_t(e) * w.N + tile * kTileRows, w.K, step * kBfCols);
  }
}

// Stages of a warp's ring.  4-bit: two, so that two CTAs fit an SM and L1 keeps
// the activations (three leave one CTA: 52 -> 73 us for one token, 8 of 128
// experts of 6144 x 2048).  BF16: three in one CTA per SM (two CTAs of two
// stages: 112 -> 121 us).
template <class SRC>
constexpr int moe_depth() { return SRC::NG > 0 || !SRC::kCopies ? 2 : 3; }
template <class SRC>
constexpr uint32_t moe_ring() { return moe_depth<SRC>() * SRC::kStage; }  // one warp's
// Shared memory after the rings: A's parts (8 warps x 16 x 16), B's sums (8
// warps x 32 rows x 8 pairs of gate and up, or 16 of one of them), C's
// accumulators (8 warps x 16 tokens x 32 rows).  The choice's scores and keys
// (8 warps x 2 x 1024) use the rings, idle then.
constexpr uint32_t kShare = 16384;
template <class SRC>
constexpr uint32_t moe_smem() { return kWarps * moe_ring<SRC>() + kShare + kWarps * moe_depth<SRC>() * 8 + 1024; }

// A unit's 32 hidden values of pair `pair` (one a lane), rows 32 ft .. of h.
template <class SRC>
__device__ __forceinline__ void store_hidden(const MoeParams& p, uint32_t pair, uint32_t ft, int lane, float v) {
  const uint32_t row = ft * kTileRows + lane;
  if (row >= p.F) v = 0.f;
  if constexpr (SRC::NG > 0) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu);
    const int k = record_exponent(m);
    const float s = v * power_of_two(k);
    const uint32_t run = ft & 3, t = uint32_t(lane) >> 3, i = 2 * run + ((uint32_t(lane) >> 2) & 1), e = lane & 3;
    uint16_t bits;
    asm("cvt.rn.f16.f32 %0, %1;" : "=h"(bits) : "f"(s));
    uint8_t* rec = p.h + (uint64_t(pair) * (p.Fp / kSub) + (ft >> 2)) * kRecord;
    *reinterpret_cast<uint16_t*>(rec + (i >> 2) * 128 + t * 32 + (i & 3) * 8 + (e & 1) * 4 + (e >> 1) * 2) = bits;
    if (lane == 0) p.hf[uint64_t(ft) * factor_pitch<4>() + pair] = power_of_two(-k);
  } else {
    uint16_t hi, lo;
    split_bf16(v, hi, lo);
    uint16_t* h = reinterpret_cast<uint16_t*>(p.h) + uint64_t(pair) * 2 * p.Fp + row;
    h[0] = hi;
    h[p.Fp] = lo;
  }
}

// Phase B: this warp's k-steps [w0, w1) of the gate and up tiles for one
// expert's n pairs from p0 on, then the unit's sums: thread i gets output i +
// 256 j (row i % 32, pair i / 32 + 8 j) as g[j] and u[j].  Up to 8 pairs take
// gate and up steps in turn, so that x comes from L1 for one of them; more take
// all gate steps, then all up steps, with one set of accumulators.
template <class SRC, int TILES, class RING, class ISSUE>
__device__ __forceinline__ void gate_up(const MoeParams& p, const Lists& L, uint32_t p0, uint32_t n, uint32_t w0,
                                        uint32_t w1, RING& ring, int lane, int warp, uint32_t magic, float* share,
                                        ISSUE& issue, float (&g)[2], float (&u)[2]) {
  const XRows<TILES> x = x_rows<TILES>(
      n, lane, [&](uint32_t b) { return p.xs + L.tok[p0 + b] * p.xs_bytes; },
      [&](uint32_t b) { return p.xf + L.tok[p0 + b]; });
  if constexpr (TILES == 1) {
    float ag[2][1][4], au[2][1][4];
    zero<1>(ag);
    zero<1>(au);
    if (w0 < w1) {
      Product<SRC, 1, 1> prod;
      prod.begin(x, w0);
#pragma unroll 1
      for (uint32_t k = w0; k < w1; ++k) {
        prod.step(ring, k, k, lane, magic, x, ag, issue);
        prod.step(ring, k, k + 1 < w1 ? k + 1 : k, lane, magic, x, au, issue);
      }
    }
    __syncthreads();  // what was in `share` is read
    put_sums<1>(share + warp * 512, lane, ag);
    put_sums<1>(share + warp * 512 + 256, lane, au);
    __syncthreads();
    const bool ok = uint32_t(warp) < n;
    g[0] = ok ? warp_sums<1>(share, kWarps, 512, lane, warp) : 0.f;
    u[0] = ok ? warp_sums<1>(share + 256, kWarps, 512, lane, warp) : 0.f;
    g[1] = u[1] = 0.f;
  } else {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      float acc[2][TILES][4];
      zero<TILES>(acc);
      if (w0 < w1) {
        Product<SRC, TILES, 1> prod;
        prod.begin(x, w0);
#pragma unroll 1
        for (uint32_t k = w0; k < w1; ++k) prod.step(ring, k, k + 1 < w1 ? k + 1 : k, lane, magic, x, acc, issue);
      }
      __syncthreads();
      put_sums<TILES>(share + warp * 512, lane, acc);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t b = warp + 8 * j;
        const float v = b < n ? warp_sums<TILES>(share, kWarps, 512, lane, b) : 0.f;
        if (i == 0)
          g[j] = v;
        else
          u[j] = v;
      }
    }
  }
}

// Phase C: the share [k0, k1) of one expert's k-steps that this warp takes,
// added to its accumulators ys[token][32 rows].  4-bit: pair c is column c of
// the MMA.  BF16: columns 2c and 2c + 1 are the parts of pair c, so one lane
// holds both sums.
template <class SRC, int TILES, class RING, class ISSUE>
__device__ __forceinline__ void down(const MoeParams& p, const Lists& L, uint32_t p0, uint32_t n, uint32_t k0,
                                     uint32_t k1, RING& ring, int lane, uint32_t magic, float* ys, ISSUE& issue) {
  constexpr bool kQ4 = SRC::NG > 0;
  const XRows<TILES> x = x_rows<TILES>(
      kQ4 ? n : 2 * n, lane,
      [&](uint32_t b) {
        return kQ4 ? p.h + uint64_t(p0 + b) * (p.Fp / kSub) * kRecord : p.h + (uint64_t(p0) * 2 + b) * p.Fp * 2;
      },
      [&](uint32_t b) { return p.hf + p0 + b; });
  float acc[2][TILES][4];
  zero<TILES>(acc);
  Product<SRC, TILES, 4> prod;
  prod.begin(x, k0);
  for (uint32_t k = k0; k < k1; ++k) prod.step(ring, k, k + 1 < k1 ? k + 1 : k, lane, magic, x, acc, issue);
  const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
#pragma unroll
  for (int nt = 0; nt < TILES; ++nt) {
#pragma unroll
    for (int i = 0; i < (kQ4 ? 2 : 1); ++i) {
      const uint32_t c = kQ4 ? 8 * nt + 2 * t + i : 4 * nt + t;
      if (c < n) {
        float* y = ys + L.tok[p0 + c] * 32 + g;
        const float w = L.w[p0 + c];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float lo = kQ4 ? acc[m][nt][i] : acc[m][nt][0] + acc[m][nt][1];
          const float hi = kQ4 ? acc[m][nt][2 + i] : acc[m][nt][2] + acc[m][nt][3];
          y[16 * m] = fmaf(w, lo, y[16 * m]);
          y[16 * m + 8] = fmaf(w, hi, y[16 * m + 8]);
        }
      }
    }
  }
  __syncwarp();  // the next expert's pairs may touch the same tokens from other lanes
}

// Phase A: units of 16 experts and a quarter of H.  Lane (g, t) takes columns
// 16 t .. 16 t + 15 of a 64-column step of rows g and g + 8 and of tokens g (and
// g + 8), straight from memory, several steps at a time.
template <bool VEC>
__device__ __forceinline__ void load16(const uint16_t* row, uint32_t c, uint32_t n, bool ok, uint32_t (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0u;
  if (!ok) return;
  if constexpr (VEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (c + 8 * h < n) {
        const uint4 u = *reinterpret_cast<const uint4*>(row + c + 8 * h);
        v[4 * h] = u.x; v[4 * h + 1] = u.y; v[4 * h + 2] = u.z; v[4 * h + 3] = u.w;
      }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (c + e < n) v[e >> 1] |= uint32_t(row[c + e]) << (16 * (e & 1));
  }
}
template <int NT, bool VEC>
__device__ __forceinline__ void router_logits(const MoeParams& p, float* share, int lane, int warp) {
  const uint32_t tiles = uint32_t(cdiv(p.E, 16)), steps = uint32_t(cdiv(p.H, kBfCols));
  const uint32_t g = uint32_t(lane) >> 2, t = uint32_t(lane) & 3;
  constexpr int U = VEC ? 4 / NT : 1;
  for (uint32_t u = blockIdx.x; u < tiles * kSplits; u += gridDim.x) {
    const uint32_t tile = u / kSplits, sp = u % kSplits, part_i = sp * kWarps + warp;
    constexpr uint32_t parts = kSplits * kWarps;
    const uint32_t k0 = uint32_t(uint64_t(steps) * part_i / parts), k1 = uint32_t(uint64_t(steps) * (part_i + 1) / parts);
    const uint32_t e0 = tile * 16 + g;
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
    for (uint32_t s0 = k0; s0 < k1; s0 += U) {
      uint32_t wg[U][8], wh[U][8], xv[U][NT][8];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t c = (s0 + i) * kBfCols + 16 * t;
        const bool in = s0 + i < k1;
        load16<VEC>(p.router + uint64_t(e0) * p.H, c, p.H, in && e0 < p.E, wg[i]);
        load16<VEC>(p.router + uint64_t(e0 + 8) * p.H, c, p.H, in && e0 + 8 < p.E, wh[i]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          load16<VEC>(p.x + uint64_t(g + 8 * nt) * p.H, c, p.H, in && g + 8 * nt < p.T, xv[i][nt]);
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_bf16_k16(acc[nt], wg[i][2 * j], wh[i][2 * j], wg[i][2 * j + 1], wh[i][2 * j + 1], xv[i][nt][2 * j],
                         xv[i][nt][2 * j + 1]);
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      *reinterpret_cast<float4*>(share + (warp * 2 + nt) * 128 + lane * 4) =
          make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
    __syncthreads();
    const uint32_t j = threadIdx.x % 16, b = threadIdx.x / 16, e = tile * 16 + j;
    if (b < p.T && e < p.E) {
      const float* src = share + (b >> 3) * 128 + ((j & 7) * 4 + ((b & 7) >> 1)) * 4 + (j >> 3) * 2 + (b & 1);
      float v = 0.f;
      for (int w = 0; w < kWarps; ++w) v += src[w * 256];
      p.logits[(uint64_t(b) * p.E + e) * kSplits + sp] = v;
    }
  }
}

// WIDE: more than 8 tokens, whose experts may have more than 8 pairs.  The
// narrow kernel is smaller by the products for those.
template <class SRC, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2) moe_kernel(const __grid_constant__ MoeParams p,
                                                          const __grid_constant__ MoeMaps maps) {
  static_assert(moe_ring<SRC>() >= kMaxE * 8, "the rings hold the scores and keys");
  constexpr int D = moe_depth<SRC>();
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // boxes are swizzled in 1024 bytes
  __shared__ Lists L;
  __shared__ Choice ch;
  __shared__ uint32_t s_flag;
  const uint32_t magic = q4_magic();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* share = reinterpret_cast<float*>(smem + kWarps * moe_ring<SRC>());
  Ring<SRC, D> ring(smem_u32(smem) + uint32_t(warp) * moe_ring<SRC>(),
                    smem_u32(smem) + kWarps * moe_ring<SRC>() + kShare + uint32_t(warp) * D * 8, p.err, lane);

  // ---- A: router logits, and x in the form that the products take
  if (p.x_vec)
    router_logits<WIDE ? 2 : 1, true>(p, share, lane, warp);
  else
    router_logits<WIDE ? 2 : 1, false>(p, share, lane, warp);
  if (p.make) {
    // from the last CTA on: the first ones have the router
    const uint32_t first = (gridDim.x - 1 - blockIdx.x) * kWarps + warp, stride = gridDim.x * kWarps;
    if constexpr (SRC::NG > 0) {
      const uint32_t recs = uint32_t(p.xs_bytes / kRecord);
      for (uint32_t i = first; i < p.T * recs; i += stride) {
        const uint32_t b = i / recs, rec = i - b * recs, c = rec * kSub + 4 * lane;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = c + e < p.H ? __uint_as_float(uint32_t(p.x[uint64_t(b) * p.H + c + e]) << 16) : 0.f;
        record_store(p.make + i * uint64_t(kRecord), p.xf + uint64_t(rec) * factor_pitch<1>() + b, v, lane);
      }
    } else {
      const uint32_t Hp = uint32_t(p.xs_bytes / 2);
      uint16_t* out = reinterpret_cast<uint16_t*>(p.make);
      for (uint32_t i = first * 32 + lane; i < p.T * Hp; i += stride * 32) {
        const uint32_t b = i / Hp, c = i - b * Hp;
        out[i] = c < p.H ? p.x[uint64_t(b) * p.H + c] : uint16_t(0);
      }
    }
  }
  bool ok = grid_barrier(p.counters, p.err, &s_flag, true);
  if (ok) {
    // ---- the choice, alike in every CTA
    for (uint32_t t = warp; t < p.T; t += kWarps) {
      if (p.E <= 128)
        choose<4>(p, t, lane, ch);
      else if (p.E <= 256)
        choose<8>(p, t, lane, ch);
      else
        choose_many(p, t, lane, reinterpret_cast<float*>(smem + warp * moe_ring<SRC>()), ch);
      weigh(p, t, lane, ch);
    }
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x < p.T * p.k) {
      if (p.ids) p.ids[threadIdx.x] = ch.e[threadIdx.x];
      if (p.weights) p.weights[threadIdx.x] = ch.w[threadIdx.x];
    }
    build_lists(p, ch, L);
    // the scores were written to the rings by ordinary stores: order them
    // before the copies that follow
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();

    // ---- B: gate and up
    const uint32_t ft_n = uint32_t(cdiv(p.F, kTileRows));
    {
      const Cuts cuts(L.active * ft_n, uint32_t(cdiv(p.H, SRC::kCols)), gridDim.x,
                      kJoinCopies / 2);  // a k-step is two copies
      Parts ahead(cuts);
      // copies left: gate and up in turn, or (many pairs) all gate, then `iup` up
      uint32_t ileft = 0, iup = 0, ia = ahead.unit / ft_n, ift = ahead.unit - ia * ft_n;
      typename SRC::Cursor cg{}, cu{};
      auto enter = [&]() {
        while (ahead.more()) {
          const uint32_t w0 = ahead.w0(warp);
          ileft = 2 * (ahead.w1(warp) - w0);
          if (ileft) {
            const uint32_t e = L.expert[ia];
            if (WIDE) iup = L.start[ia + 1] - L.start[ia] > 8 ? ileft / 2 : 0;
            cg = expert_at<SRC>(p, maps, 0, e, ift, w0);
            cu = expert_at<SRC>(p, maps, 1, e, ift, w0);
          }
          ahead.next();
          if (++ift == ft_n) {
            ift = 0;
            ++ia;
          }
          if (ileft) return;
        }
      };
      auto issue = [&](uint32_t slot) {
        if (ileft) {
          if (WIDE && iup ? ileft <= iup : ileft & 1)
            ring.refill(slot, cu, lane);
          else
            ring.refill(slot, cg, lane);
          if (--ileft == 0) enter();
        }
      };
      enter();
      for (uint32_t i = 0; i < D; ++i) issue((ring.slot + i) % D);
      Parts s(cuts);
      uint32_t a = s.unit / ft_n, ft = s.unit - a * ft_n;
      for (bool first_part = true; s.more(); s.next(), first_part = false) {
        const uint32_t p0 = L.start[a], n = L.start[a + 1] - p0, w0 = s.w0(warp), w1 = s.w1(warp);
        float g[2], u[2];
        if (!WIDE || n <= 8)
          gate_up<SRC, 1>(p, L, p0, n, w0, w1, ring, lane, warp, magic, share, issue, g, u);
        else if constexpr (WIDE)
          gate_up<SRC, 2>(p, L, p0, n, w0, w1, ring, lane, warp, magic, share, issue, g, u);
        auto hidden = [&](int j, float gv, float uv) {
          const uint32_t c = warp + 8 * j;
          if (c >= n) return;
          store_hidden<SRC>(p, p0 + c, ft, lane, gv / (1.f + expf(-gv)) * uv);
          if (ft + 1 == ft_n)  // zeros up to the rows' padded end
            for (uint32_t f = ft_n; f < p.Fp / kTileRows; ++f) store_hidden<SRC>(p, p0 + c, f, lane, 0.f);
        };
        if (s.whole()) {
#pragma unroll 1
          for (int j = 0; j < 2; ++j) hidden(j, j ? g[1] : g[0], j ? u[1] : u[0]);
        } else {
          // thread i's four values are i + 256 q: gate of pairs 0..7, gate of 8..15, then up
          float gs[2];
          join_parts(
              cuts, s, first_part, p.part, kPartFloats, p.counters + 8, kPartFloats, &s_flag,
              [&](uint32_t i) { return i < 256 ? g[0] : i < 512 ? g[1] : i < 768 ? u[0] : u[1]; },
              [&](uint32_t i, float v) {
                if (i < 256)
                  gs[0] = v;
                else if (i < 512)
                  gs[1] = v;
                else
                  hidden(i < 768 ? 0 : 1, i < 768 ? gs[0] : gs[1], v);
              });
        }
        if (++ft == ft_n) {
          ft = 0;
          ++a;
        }
      }
    }

    // ---- C: down and the weighted sum.  A unit's k-steps are those of all
    // chosen experts, one expert after the other.
    {
      const uint32_t steps = uint32_t(cdiv(p.F, SRC::kCols));
      // a k-step is one copy, but half of a join's cost is taken: a run of copies is
      // longer here by each expert's beginning and end (us with whole / half the cost,
      // 6 of 12 4-bit experts: 512 x 512, 4 tokens 20.6 / 18.7; 461 x 474, 16 tokens 30.9 / 28.3;
      // with a quarter, 2 of 8 BF16 ones of 1024 x 512, 1 token: 13.7 -> 17.5)
      const Cuts cuts(uint32_t(cdiv(p.H, kTileRows)), L.active * steps, gridDim.x, kJoinCopies / 2);
      // the cursor's place: ileft k-steps to expert ia's or the warp's end, irest
      // after those
      Parts ahead(cuts);
      uint32_t ia = 0, iunit = 0, ileft = 0, irest = 0;
      typename SRC::Cursor cd{};
      auto tile = [&](uint32_t k) {
        ileft = irest < steps - k ? irest : steps - k;
        irest -= ileft;
        cd = expert_at<SRC>(p, maps, 2, L.expert[ia], iunit, k);
      };
      auto enter = [&]() {
        for (; ahead.more(); ahead.next()) {
          const uint32_t w0 = ahead.w0(warp);
          irest = ahead.w1(warp) - w0;
          iunit = ahead.unit;
          if (irest) {
            ia = w0 / steps;
            tile(w0 - ia * steps);
            ahead.next();
            return;
          }
        }
      };
      auto issue = [&](uint32_t slot) {
        if (ileft) {
          ring.refill(slot, cd, lane);
          if (--ileft == 0) {
            if (irest) {
              ++ia;
              tile(0);
            } else {
              enter();
            }
          }
        }
      };
      enter();
      for (uint32_t i = 0; i < D; ++i) issue((ring.slot + i) % D);
      ok = grid_barrier(p.counters + 1, p.err, &s_flag, false);
      if (ok) {
        bool first_part = true;
        for (Parts s(cuts); s.more(); s.next(), first_part = false) {
          float* ys = share + warp * (kMaxT * 32);
          __syncthreads();  // the previous unit's accumulators are read
          for (uint32_t i = lane; i < p.T * 32; i += 32) ys[i] = 0.f;
          __syncwarp();
          const uint32_t w1 = s.w1(warp);
          uint32_t k = s.w0(warp), a = k / steps, k0 = k - a * steps;
          for (; k < w1; ++a, k0 = 0) {
            const uint32_t k1 = w1 - k < steps - k0 ? k0 + (w1 - k) : steps;
            const uint32_t p0 = L.start[a], n = L.start[a + 1] - p0;
            if constexpr (SRC::NG > 0) {
              if (!WIDE || n <= 8)
                down<SRC, 1>(p, L, p0, n, k0, k1, ring, lane, magic, ys, issue);
              else if constexpr (WIDE)
                down<SRC, 2>(p, L, p0, n, k0, k1, ring, lane, magic, ys, issue);
            } else {
              if (n <= 4)
                down<SRC, 1>(p, L, p0, n, k0, k1, ring, lane, magic, ys, issue);
              else if (!WIDE || n <= 8)
                down<SRC, 2>(p, L, p0, n, k0, k1, ring, lane, magic, ys, issue);
              else if constexpr (WIDE)
                down<SRC, 4>(p, L, p0, n, k0, k1, ring, lane, magic, ys, issue);
            }
            k += k1 - k0;
          }
          __syncthreads();
          // output i: row i % 32 of the unit, token i / 32
          auto value = [&](uint32_t i) {
            float v = 0.f;
            for (int w = 0; w < kWarps; ++w) v += share[w * (kMaxT * 32) + i];
            return v;
          };
          auto store = [&](uint32_t i, float v) {
            const uint32_t row = s.unit * 32 + i % 32, b = __float_as_uint(v);
            if (row < p.H)
              p.y[uint64_t(i / 32) * p.H + row] =
                  (b & 0x7FFFFFFFu) > 0x7F800000u ? uint16_t(0x7FC0) : uint16_t((b + 0x7FFFu + ((b >> 16) & 1u)) >> 16);
          };
          if (s.whole()) {
            for (uint32_t i = threadIdx.x; i < p.T * 32; i += kThreads) store(i, value(i));
          } else {
            join_parts(cuts, s, first_part, p.part + 2 * uint64_t(gridDim.x) * kPartFloats, kPartFloats,
                       p.counters + 8 + kMaxGrid, p.T * 32, &s_flag, value, store);
          }
        }
      } else {
        ring.abandon();
      }
    }
  }
  // the last CTA to finish leaves the counters at zero for their next launch:
  // after a barrier that ran out also those of joins that not every CTA came to
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const uint32_t done = atomicAdd(p.counters + 2, ok ? 1u : 0x10001u) + (ok ? 1u : 0x10001u);
    if ((done & 0xFFFFu) == gridDim.x) {
      __threadfence();
      for (uint32_t i = 0; i < (done >> 16 ? kSlotWords : 3u); ++i) p.counters[i] = 0u;
    }
  }
}

template <class SRC, bool WIDE>
int launch_moe_as(MoeParams& p, const MoeMaps& maps, int dev, cudaStream_t s) {
  static std::atomic<int> cache[64];
  auto kern = moe_kernel<SRC, WIDE>;
  constexpr uint32_t smem = moe_smem<SRC>();
  int per_sm = cache[dev].load(std::memory_order_acquire);
  if (!per_sm) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess)
      return map_cuda(cudaGetLastError());
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, smem);
    if (e != cudaSuccess) return map_cuda(e);
    if (per_sm < 1) return WCOMP_EUNSUPPORTED;
    cache[dev].store(per_sm, std::memory_order_release);
  }
  const uint32_t grid = std::min(uint32_t(per_sm * sm_count(dev)), kMaxGrid);
  void* args[] = {&p, const_cast<MoeMaps*>(&maps)};
  const cudaError_t e =
      cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kern), dim3(grid), dim3(kThreads), args, smem, s);
  count_launches(1);
  return map_cuda(e == cudaSuccess ? cudaGetLastError() : e);
}

template <class SRC>
int launch_moe(MoeParams& p, const MoeMaps& maps, int dev, cudaStream_t s) {
  return p.T > 8 ? launch_moe_as<SRC, true>(p, maps, dev, s) : launch_moe_as<SRC, false>(p, maps, dev, s);
}

// Boxes of 32 rows x 64 columns of a row-major BF16 matrix, 128-byte swizzled.
bool box_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols) {
  const EncodeTiledFn f = tensor_map_encoder();
  if (!f || cols % 8 || (reinterpret_cast<uintptr_t>(base) & 15) || rows >= (uint64_t(1) << 31)) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols * 2};
  const cuuint32_t box[2] = {uint32_t(kBfCols), uint32_t(kTileRows)};
  const cuuint32_t es[2] = {1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

WCOMP_DEBUG_HOOKS(debug_hooks_moe)
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
  p.x = a->d_x;
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
  p.x_vec = p.H % 8 == 0 && aligned(a->d_x, 16) && aligned(a->d_router, 16);
  MoeMaps maps;
  memset(&maps, 0, sizeof(maps));
  bool mapped = !q4;
  for (int i = 0; i < 3; ++i) {
    Weights& t = p.w[i];
    t.N = i == 2 ? p.H : p.F;
    t.K = i == 2 ? p.F : p.H;
    t.p = q4 ? q[i]->d : reinterpret_cast<const uint8_t*>(w[i]);
    t.expert_bytes = q4 ? q[i]->matrix_bytes() : 0;
    if (!q4) mapped = mapped && box_map(&maps.m[i], w[i], uint64_t(p.E) * t.N, t.K);
  }
  // x's form for the products: records, or BF16 rows of whole 64-column steps
  // that start on 32-byte boundaries
  const uint64_t Hp = q4 ? cdiv(p.H, kQ4Cols) * kQ4Cols : cdiv(p.H, kBfCols) * kBfCols;
  const bool make = q4 || Hp != p.H || !aligned(a->d_x, 32);
  p.xs_bytes = 2 * Hp;
  auto round = [](uint64_t b) { return (b + 255) & ~uint64_t(255); };
  const uint64_t pairs = uint64_t(p.T) * p.k;
  const uint64_t b_log = round(uint64_t(4) * kSplits * p.T * p.E), b_h = round(pairs * p.Fp * (q4 ? 2 : 4)),
                 b_hf = q4 ? round(uint64_t(p.Fp) / 32 * factor_pitch<4>() * 4) : 0,
                 b_part = uint64_t(2) * 2 * kMaxGrid * kPartFloats * sizeof(float),
                 b_x = make ? round(p.T * p.xs_bytes) : 0, b_xf = q4 ? round(Hp / kSub * factor_pitch<1>() * 4) : 0;
  int st = work_error(dev, &p.err);
  if (st == WCOMP_OK) st = work_slot(dev, s, &p.counters);
  if (st != WCOMP_OK) return st;
  const uint64_t b_count = p.counters ? 0 : kSlotWords * sizeof(uint32_t);
  uint8_t* ws = nullptr;
  e = pool_alloc(reinterpret_cast<void**>(&ws), b_log + b_h + b_hf + b_part + b_x + b_xf + b_count, s);
  if (e != cudaSuccess) return map_cuda(e);
  uint8_t* at = ws;
  auto take = [&](uint64_t bytes) {
    uint8_t* r = at;
    at += bytes;
    return r;
  };
  p.logits = reinterpret_cast<float*>(take(b_log));
  p.h = take(b_h);
  p.hf = reinterpret_cast<float*>(take(b_hf));
  p.part = reinterpret_cast<float*>(take(b_part));
  p.make = make ? take(b_x) : nullptr;
  p.xf = reinterpret_cast<float*>(take(b_xf));
  p.xs = make ? p.make : reinterpret_cast<const uint8_t*>(a->d_x);
  if (!p.counters) {
    p.counters = reinterpret_cast<uint32_t*>(take(b_count));
    st = map_cuda(cudaMemsetAsync(p.counters, 0, b_count, s));
  }
  if (st == WCOMP_OK) {
    if (!q4)
      st = mapped ? launch_moe<BfSrc<true>>(p, maps, dev, s) : launch_moe<BfSrc<false>>(p, maps, dev, s);
    else if (q[0]->ng == 1)
      st = launch_moe<Q4Src<1>>(p, maps, dev, s);
    else if (q[0]->ng == 2)
      st = launch_moe<Q4Src<2>>(p, maps, dev, s);
    else
      st = launch_moe<Q4Src<4>>(p, maps, dev, s);
  }
  cudaFreeAsync(ws, s);
  return st;
}
