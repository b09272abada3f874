// Writing, reading and evicting from the 4-bit key/value cache.
#include <algorithm>
#include <new>
#include <type_traits>

#include "cluster.cuh"
#include "kv4.cuh"
#include "q4_rule.cuh"

namespace wc {
namespace {

constexpr int kThreads = 128;  // 256: 8% slower

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

// A row of keys or values is handled by D / 8 neighbouring lanes, lane u the columns
// 8 u .. 8 u + 7; four of them share a group.  A warp takes `span` rows of the call,
// whose places its lanes look up side by side, and kHeads heads of each: kLanes at a
// time, STEPS of them with the loads of their keys and values in flight together.
// Instructions bound the writing, 102 for 8 columns, some 60 of them their codes and
// scale, and the places' look-up where many sequences have a few rows each.  65536 rows of 8 heads, one look-up for
// four rows or (for every row), and the share of the copy rate:
//   columns  write                 read
//    64       38 (45) us  0.66      33 (37) us  0.77
//   128       68 (84)     0.75      58 (64)     0.87
//   256      130 (161)    0.78     110 (119)    0.92
// Four steps in flight leave room for fewer warps: 88 us for 75 at 128 columns.  The least
// numbers of blocks keep the compiler at the registers of these figures (56, not 72).
template <int D, int STEPS>
struct Items {
  static constexpr int kPer = D / 8;
  static constexpr int kLanes = 32 / kPer;
  static constexpr int kHeads = kLanes * STEPS;
};

// Quantise 8 columns, whose group's other columns the three neighbouring lanes have.
// `w` gets the codes, 4 bits each; returns the scale's bits.
__device__ __forceinline__ uint32_t quantise8(const uint32_t (&v)[4], uint32_t& w) {
  uint32_t m = abs_max2(abs_max2(v[0], v[1]), abs_max2(v[2], v[3]));
  m = abs_max2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = abs_max2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  m = abs_max2(m, m >> 16) & 0x7FFFu;
  const uint32_t bits = scale_of(m);
  const float s = bf16_value(bits);
  if (s >= 0x1p-100f) {
    // code_fast for two columns at a time
    const float rs = reciprocal(s);
    const uint64_t rs2 = pair(rs, rs), snap = pair(kSnap, kSnap), round = pair(kRound - kSnap, kRound - kSnap);
    w = 0u - kBase * 0x11111111u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t c = add2(fma2(pair(bf16_lo(v[i]), bf16_hi(v[i])), rs2, snap), round);
      w += uint32_t(c) * (1u << (8 * i)) + uint32_t(c >> 32) * (16u << (8 * i));
    }
  } else {
    w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w |= code_slow(bf16_lo(v[i]), s) << (8 * i) | code_slow(bf16_hi(v[i]), s) << (8 * i + 4);
  }
  return bits;
}

// The words of a value row hold four columns of two groups each: lanes u and u ^ 4
// (groups 2 a and 2 a + 1) exchange halves.  In: the lane's own 8 columns; out: the
// word at `index` of the row.  And back: the exchange is its own inverse.
__device__ __forceinline__ uint32_t value_word(uint32_t w, uint32_t u) {
  const uint32_t other = __shfl_xor_sync(0xffffffffu, w, 4);
  return (u & 4) ? prmt(other, w, 0x7632) : prmt(w, other, 0x5410);
}
template <int D>
__device__ __forceinline__ uint32_t key_index(uint32_t u) {
  return (u & 3) * Kv<D>::G + (u >> 2);
}
template <int D>
__device__ __forceinline__ uint32_t value_index(uint32_t u) {
  return (2 * (u & 3) + ((u >> 2) & 1)) * (Kv<D>::G / 2) + (u >> 3);
}

struct Rows {
  const uint16_t* p;
  int64_t row, head;
  int vec;  // rows are 16-byte aligned
};

// The place of row i: its page and the token in it.  Page -1: there is none; -2: the
// row is no sequence's.
__device__ __forceinline__ int row_place(const KvSeqs& s, int64_t i, uint32_t& t) {
  const int b = kv_sequence(s, i);
  if (b < 0) return -2;
  const int64_t pos = kv_position(s, b, i, kv_length(s, b));
  t = uint32_t(pos) % kPage;
  return pos < 0 ? -1 : kv_page(s, b, int(pos / kPage));
}
// The first row and head of a warp's unit: `rounds` units have the same rows.
__device__ __forceinline__ int64_t unit_rows(int64_t unit, uint32_t rounds, uint32_t& round) {
  if (rounds == 1) {
    round = 0;
    return unit;
  }
  const int64_t i = (unit >> 32) ? unit / rounds : int64_t(uint32_t(unit) / rounds);
  round = uint32_t(unit - i * rounds);
  return i;
}

template <int D, int STEPS>
__global__ void __launch_bounds__(kThreads, STEPS == 1 ? 10 : 9) kv4_append_kernel(KvSeqs s, uint8_t* cache, Rows k, Rows v, int64_t T,
                                                              uint32_t rounds, uint32_t span) {
  using I = Items<D, STEPS>;
  using L = Kv<D>;
  const uint32_t lane = threadIdx.x % 32, u = lane % I::kPer;
  const uint32_t key_byte = 4 * key_index<D>(u), value_byte = 4 * value_index<D>(u);
  const int64_t units = (T + span - 1) / span * rounds;
  for (int64_t unit = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; unit < units;
       unit += int64_t(gridDim.x) * (kThreads / 32)) {
    uint32_t round;
    const int64_t i0 = unit_rows(unit, rounds, round) * span;
    const uint32_t h0 = round * I::kHeads + lane / I::kPer, rows = uint32_t(min(int64_t(span), T - i0));
    uint32_t its = 0;
    const int it = lane < rows ? row_place(s, i0 + lane, its) : -2;
#pragma unroll 1
    for (uint32_t i = 0; i < rows; ++i) {
      const int page = __shfl_sync(0xffffffffu, it, i);
      const uint32_t t = __shfl_sync(0xffffffffu, its, i);
      if (page < 0) continue;
      uint32_t x[2][STEPS][4];
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const Rows& r = part ? v : k;
        const uint16_t* p = r.p + (i0 + i) * r.row + h0 * r.head + 8 * u;
        if (r.vec) {
#pragma unroll
          for (int j = 0; j < STEPS; ++j, p += I::kLanes * r.head) {
            const uint4 y = h0 + j * I::kLanes < s.heads ? ld_stream_v4(p) : make_uint4(0, 0, 0, 0);
            x[part][j][0] = y.x; x[part][j][1] = y.y; x[part][j][2] = y.z; x[part][j][3] = y.w;
          }
        } else {
#pragma unroll
          for (int j = 0; j < STEPS; ++j, p += I::kLanes * r.head)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[part][j][e] = h0 + j * I::kLanes < s.heads ? p[2 * e] | uint32_t(p[2 * e + 1]) << 16 : 0u;
        }
      }
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        uint8_t* half = cache + (uint64_t(uint32_t(page)) * s.heads + h0) * L::kBlock + part * L::kHalf;
        uint8_t* codes = half + L::at(t, part ? value_byte : key_byte);
        uint8_t* scales = half + L::scale(t, u >> 2);
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
          uint32_t w;
          const uint32_t scale = quantise8(x[part][j], w);  // every lane takes part in the exchanges
          if (part) w = value_word(w, u);
          if (h0 + j * I::kLanes >= s.heads) continue;
          *reinterpret_cast<uint32_t*>(codes + j * I::kLanes * L::kBlock) = w;
          if ((u & 3) == 0) *reinterpret_cast<uint16_t*>(scales + j * I::kLanes * L::kBlock) = uint16_t(scale);
        }
      }
    }
  }
  kv_check_starts(s, T, blockIdx.x * kThreads + threadIdx.x, gridDim.x * kThreads);
}

// Eight codes times a scale, in pairs of BF16: a code under the exponent of 128 is 128
// + c, less 136 exactly c - 8, and the product is rounded once.
__device__ __forceinline__ uint4 values8(uint32_t w, uint32_t scale) {
  const uint32_t s = prmt(scale, scale, 0x1010);
  uint32_t x[4];  // columns i and i + 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(x[i]) : "r"(0x43084308u));
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(x[i]) : "r"(s));
  }
  return make_uint4(prmt(x[0], x[1], 0x5410), prmt(x[2], x[3], 0x5410), prmt(x[0], x[1], 0x7632), prmt(x[2], x[3], 0x7632));
}

template <int D, int STEPS>
__global__ void __launch_bounds__(kThreads, 12) kv4_read_kernel(KvSeqs s, const uint8_t* cache, uint16_t* k, uint16_t* v,
                                                            int64_t T, uint32_t rounds, uint32_t span, int vec) {
  using I = Items<D, STEPS>;
  using L = Kv<D>;
  const uint32_t lane = threadIdx.x % 32, u = lane % I::kPer;
  const uint32_t key_byte = 4 * key_index<D>(u), value_byte = 4 * value_index<D>(u);
  const int64_t units = (T + span - 1) / span * rounds;
  for (int64_t unit = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; unit < units;
       unit += int64_t(gridDim.x) * (kThreads / 32)) {
    uint32_t round;
    const int64_t i0 = unit_rows(unit, rounds, round) * span;
    const uint32_t h0 = round * I::kHeads + lane / I::kPer, rows = uint32_t(min(int64_t(span), T - i0));
    uint32_t its = 0;
    const int it = lane < rows ? row_place(s, i0 + lane, its) : -2;
#pragma unroll 1
    for (uint32_t i = 0; i < rows; ++i) {
      const int page = __shfl_sync(0xffffffffu, it, i);
      const uint32_t t = __shfl_sync(0xffffffffu, its, i);
      if (page < -1) continue;
      uint32_t w[2][STEPS], scale[2][STEPS];
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const uint8_t* half = cache + (uint64_t(uint32_t(page)) * s.heads + h0) * L::kBlock + part * L::kHalf;
        const uint8_t* codes = half + L::at(t, part ? value_byte : key_byte);
        const uint8_t* scales = half + L::scale(t, u >> 2);
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
          w[part][j] = 0x88888888u;
          scale[part][j] = 0;
          if (page < 0 || h0 + j * I::kLanes >= s.heads) continue;
          w[part][j] = *reinterpret_cast<const uint32_t*>(codes + j * I::kLanes * L::kBlock);
          scale[part][j] = *reinterpret_cast<const uint16_t*>(scales + j * I::kLanes * L::kBlock);
        }
      }
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        uint16_t* p = (part ? v : k) + ((i0 + i) * s.heads + h0) * D + 8 * u;
#pragma unroll
        for (int j = 0; j < STEPS; ++j, p += I::kLanes * D) {
          const uint4 x = values8(part ? value_word(w[part][j], u) : w[part][j], scale[part][j]);
          if (h0 + j * I::kLanes >= s.heads) continue;
          if (vec) {
            *reinterpret_cast<uint4*>(p) = x;
          } else {
            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = uint16_t(y[e / 2] >> (16 * (e % 2)));
          }
        }
      }
    }
  }
  kv_check_starts(s, T, blockIdx.x * kThreads + threadIdx.x, gridDim.x * kThreads);
}

// ---------------------------------------------------------------------------
// Eviction: a block chooses the tokens of one sequence and head; then blocks copy
// 64 kept tokens each.
// ---------------------------------------------------------------------------
struct EvictArgs {
  KvSeqs s;
  const float* mass;
  float* mass_out;
  const int32_t* table_out;
  int32_t* lengths_out;
  int32_t* kept;  // [B, heads, keep]
  uint8_t* cache;
  int width_out, keep, recent;
};

constexpr int kChoose = 512, kChooseWarps = kChoose / 32;
constexpr int kHeld = 16;   // keys that a thread holds in registers, 8192 a block,
constexpr int kShared = 22; // and in shared memory, 11264 more
constexpr int kMaxTeam = 8; // blocks that share a sequence and head

// A mass as a number that orders as it does: NaN lowest, -0 and 0 alike.
__device__ __forceinline__ uint32_t mass_key(float m) {
  const uint32_t u = __float_as_uint(m + 0.f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The tokens of one sequence and head that are kept: one block, or a cluster of
// them for long sequences.  A warp has a run of consecutive tokens, their keys in
// registers as far as those go, so a step of the search for the last key taken is
// comparisons and one sum over the block: two bits of the key a step.  (A radix
// selection took 45 us for 256 sequences and heads of up to 16384 tokens: few
// exponents, so its counters in shared memory are fought over.)
struct Choose {
  uint32_t sums[2][kChooseWarps][3];  // by the parity of the step
  uint32_t team[2][3];                // this block's
  uint32_t below[2][kChooseWarps];
  uint32_t keys[kShared][kChoose];
};

__global__ void __launch_bounds__(kChoose, 2) kv4_choose_kernel(EvictArgs a, uint32_t team) {
  __shared__ Choose sh;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = team > 1 ? cluster_rank() : 0;
  const int64_t unit = blockIdx.x / team;
  const int b = int(unit / a.s.heads);
  const int n = kv_length(a.s, b);
  const int m = min(n, a.keep);
  const float* mass = a.mass + unit * (int64_t(a.s.width) * kPage);
  float* mass_out = a.mass_out + unit * (int64_t(a.width_out) * kPage);
  int32_t* kept = a.kept + unit * a.keep;
  if (unit % a.s.heads == 0 && tid == 0 && rank == 0) a.lengths_out[b] = m;
  const bool all = m == n;
  const int n0 = all ? 0 : n - a.recent;              // tokens to choose from; those behind are kept
  const uint32_t want = all ? 0 : uint32_t(a.keep - a.recent);
  // this warp's tokens: i0 + 32 k + lane below i1
  const int run = ((n + 31) / 32 + int(team * kChooseWarps) - 1) / int(team * kChooseWarps) * 32;
  const int64_t start = int64_t(rank * kChooseWarps + warp) * run;
  const int i0 = int(min(int64_t(n), start)), i1 = min(n, i0 + run), steps = run / 32;
  // keys of the tokens to choose from, others 0: nothing that is searched for is
  uint32_t held[kHeld];
  auto load = [&](int k) {
    const int i = i0 + 32 * k + int(lane);
    return i < min(i1, n0) ? mass_key(mass[i]) : 0u;
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k) held[k] = load(k);
#pragma unroll 8
  for (int k = kHeld; k < min(steps, kHeld + kShared); ++k) sh.keys[k - kHeld][tid] = load(k);
  auto key_at = [&](int k) {  // beyond the registers
    return k < kHeld + kShared ? sh.keys[k - kHeld][tid] : load(k);
  };
  auto candidates = [&](auto f) {
#pragma unroll
    for (int k = 0; k < kHeld; k += 4)
      if (k < steps) {
        f(held[k]);
        f(held[k + 1]);
        f(held[k + 2]);
        f(held[k + 3]);
      }
    const int shared = min(steps, kHeld + kShared);
#pragma unroll 8
    for (int k = kHeld; k < shared; ++k) f(sh.keys[k - kHeld][tid]);
#pragma unroll 4
    for (int k = shared; k < steps; ++k) f(load(k));
  };
  // the sum of three counts over all tokens
  uint32_t parity = 0;
  auto sum3 = [&](uint32_t (&c)[3]) {
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      c[j] = __reduce_add_sync(0xffffffffu, c[j]);
      if (lane == 0) sh.sums[parity][warp][j] = c[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 3; ++j)
      c[j] = __reduce_add_sync(0xffffffffu, lane < kChooseWarps ? sh.sums[parity][lane][j] : 0u);
    if (team > 1) {
      if (tid < 3) sh.team[parity][tid] = c[tid];
      cluster_sync();
#pragma unroll
      for (int j = 0; j < 3; ++j)
        c[j] = __reduce_add_sync(0xffffffffu, lane < team ? cluster_lds_u32(smem_u32(&sh.team[parity][j]), lane) : 0u);
    }
    parity ^= 1;
  };
  // the largest key that at least `want` tokens reach, or one that just `want` do
  uint32_t key = 0, reach = 0;
  if (want) {
    for (int shift = 30; shift >= 0 && reach != want; shift -= 2) {
      uint32_t c[3] = {0, 0, 0};
      candidates([&](uint32_t k) {
#pragma unroll
        for (uint32_t j = 0; j < 3; ++j) c[j] += k >= (key | (j + 1) << shift);
      });
      sum3(c);
      const uint32_t digit = c[2] >= want ? 3u : c[1] >= want ? 2u : c[0] >= want ? 1u : 0u;
      key |= digit << shift;
      if (digit) reach = c[digit - 1];
    }
  }
  // above it all are taken; of those that equal it, the first ones
  const bool some = want != 0;
  uint32_t above = 0, equal = 0;
  auto count = [&](int i, uint32_t k) {
    const bool in = i < min(i1, n0) && some;
    above += __popc(__ballot_sync(0xffffffffu, (i < i1 && i >= n0) || (in && k > key)));
    equal += __popc(__ballot_sync(0xffffffffu, in && k == key));
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (k < steps) count(i0 + 32 * k + int(lane), held[k]);
#pragma unroll 8
  for (int k = kHeld; k < steps; ++k) count(i0 + 32 * k + int(lane), key_at(k));
  // sums over the warps before this one, and the number taken above the key
  uint32_t before[2] = {0, 0}, taken;
  {
    if (lane == 0) {
      sh.below[0][warp] = above;
      sh.below[1][warp] = equal;
    }
    uint32_t c[3] = {lane == 0 ? above : 0u, lane == 0 ? equal : 0u, 0u};
    uint32_t own[2];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t v = lane < kChooseWarps ? sh.below[j][lane] : 0u;
      own[j] = __reduce_add_sync(0xffffffffu, v);
      before[j] = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0u);
    }
    if (team > 1) {
      if (tid < 2) sh.team[parity][tid] = own[tid];
      cluster_sync();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t v = lane < team ? cluster_lds_u32(smem_u32(&sh.team[parity][j]), lane) : 0u;
        before[j] += __reduce_add_sync(0xffffffffu, lane < rank ? v : 0u);
        c[j] = __reduce_add_sync(0xffffffffu, v);
      }
    } else {
      c[0] = own[0];
    }
    taken = c[0];
  }
  const uint32_t ties = some ? uint32_t(m) - taken : 0u;  // of the equal ones, the first `ties`
  uint32_t seen = before[1], place = before[0] + min(before[1], ties);
  auto emit = [&](int i, uint32_t k, float x) {
    const bool in = i < min(i1, n0) && some;
    const bool tie = in && k == key;
    const uint32_t tied = __ballot_sync(0xffffffffu, tie), lower = (1u << lane) - 1u;
    const bool take = (i < i1 && i >= n0) || (in && k > key) || (tie && seen + __popc(tied & lower) < ties);
    const uint32_t takes = __ballot_sync(0xffffffffu, take);
    if (take) {
      const uint32_t to = place + __popc(takes & lower);
      kept[to] = i;
      mass_out[to] = x;
    }
    seen += __popc(tied);
    place += __popc(takes);
  };
  // eight masses at a time, before what is done with them waits for the first
  float x[8];
  auto masses = [&](int k) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + 32 * (k + j) + int(lane);
      x[j] = i < i1 ? mass[i] : 0.f;
    }
  };
#pragma unroll
  for (int k = 0; k < kHeld; k += 8)
    if (k < steps) {
      masses(k);
#pragma unroll
      for (int j = 0; j < 8; ++j) emit(i0 + 32 * (k + j) + int(lane), held[k + j], x[j]);
    }
  for (int k = kHeld; k < steps; k += 8) {
    masses(k);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k + j < steps) emit(i0 + 32 * (k + j) + int(lane), key_at(k + j), x[j]);
  }
  for (int i = m + int(rank * kChoose + tid); i < a.keep; i += int(team * kChoose)) kept[i] = -1;
  for (int i = m + int(rank * kChoose + tid); i < a.width_out * kPage; i += int(team * kChoose)) mass_out[i] = 0.f;
  if (team > 1) cluster_sync();  // a block's shared memory stays while others read it
}

constexpr int kMove = 128;
template <int D>
__global__ void __launch_bounds__(kMove, D == 256 ? 5 : 10) kv4_move_kernel(EvictArgs a) {
  using L = Kv<D>;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ int64_t s_src[kPage];  // the block's source and the token in it, or
  constexpr int64_t kNothing = -1, kMissing = -2;  // no token; one of a page that does not exist
  __shared__ uint32_t s_at[kPage];
  const int64_t tiles = (a.keep + kPage - 1) / kPage;
  const int64_t units = int64_t(a.s.B) * a.s.heads * tiles;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t bh = unit / tiles;
    const int tile = int(unit % tiles), b = int(bh / a.s.heads), h = int(bh % a.s.heads);
    bool missing = false;
    __syncthreads();
    if (threadIdx.x < kPage) {
      const int i = tile * kPage + int(threadIdx.x);
      const int pos = i < a.keep ? a.kept[bh * a.keep + i] : -1;
      const int page = pos < 0 ? -1 : kv_page(a.s, b, pos / kPage);
      missing = pos >= 0 && page < 0;
      s_src[threadIdx.x] = pos < 0 ? kNothing : missing ? kMissing : (int64_t(page) * a.s.heads + h) * L::kBlock;
      s_at[threadIdx.x] = uint32_t(pos) % kPage;
    }
    missing = __syncthreads_or(missing);
    if (a.kept[bh * a.keep + tile * kPage] < 0) continue;  // a shorter sequence: nothing here, no page needed
    const int out = a.table_out[int64_t(b) * a.width_out + tile];
    if (uint32_t(out) >= a.s.pages) {
      if (threadIdx.x == 0) kv_bad(a.s.err);
      continue;
    }
    uint8_t* dst = a.cache + (uint64_t(out) * a.s.heads + h) * L::kBlock;
    // every load of a round is in flight before the first store
    constexpr int kPieces = 2 * L::kRow / 16;  // 16-byte pieces of a token's keys and values
    constexpr int kRounds = kPage * kPieces / kMove, kScaleRounds = kPage * 2 * L::G / kMove;
    uint4 x[kRounds];
    uint16_t y[kScaleRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const uint32_t j = threadIdx.x + k * kMove, t = j / kPieces, piece = j % kPieces;
      const uint32_t part = piece / (kPieces / 2) * L::kHalf, byte = piece % (kPieces / 2) * 16;
      if (s_src[t] >= 0) x[k] = *reinterpret_cast<const uint4*>(a.cache + s_src[t] + part + L::at(s_at[t], byte));
    }
#pragma unroll
    for (int k = 0; k < kScaleRounds; ++k) {
      const uint32_t j = threadIdx.x + k * kMove, t = j % kPage, g = j / kPage;
      if (s_src[t] >= 0)
        y[k] = *reinterpret_cast<const uint16_t*>(a.cache + s_src[t] + g / L::G * L::kHalf + L::scale(s_at[t], g % L::G));
    }
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const uint32_t j = threadIdx.x + k * kMove, t = j / kPieces, piece = j % kPieces;
      const uint32_t part = piece / (kPieces / 2) * L::kHalf, byte = piece % (kPieces / 2) * 16;
      if (s_src[t] >= 0) *reinterpret_cast<uint4*>(dst + part + L::at(t, byte)) = x[k];
    }
#pragma unroll
    for (int k = 0; k < kScaleRounds; ++k) {
      const uint32_t j = threadIdx.x + k * kMove, t = j % kPage, g = j / kPage;
      if (s_src[t] >= 0) *reinterpret_cast<uint16_t*>(dst + g / L::G * L::kHalf + L::scale(t, g % L::G)) = y[k];
    }
    if (!missing) continue;
    // rows of zeros in their places
#pragma unroll 1
    for (uint32_t j = threadIdx.x; j < kPage * kPieces; j += kMove) {
      const uint32_t t = j / kPieces, piece = j % kPieces, part = piece / (kPieces / 2) * L::kHalf;
      if (s_src[t] != kMissing) continue;
      *reinterpret_cast<uint4*>(dst + part + L::at(t, piece % (kPieces / 2) * 16)) =
          make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
      static_assert(kPieces == 2 * L::G, "as many scales as pieces");
      *reinterpret_cast<uint16_t*>(dst + piece / L::G * L::kHalf + L::scale(t, piece % L::G)) = 0;
    }
  }
}

bool on_device(const wcomp_kv4* c) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == c->device;
}

constexpr uint32_t kMaxSpan = 4;  // rows of a warp, once the GPU has 64 units an SM

uint32_t grid_of(int64_t blocks, int dev) {
  return uint32_t(std::max<int64_t>(1, std::min<int64_t>(blocks, int64_t(sm_count(dev)) * 64)));
}

bool rows_vec(const uint16_t* p, int64_t row, int64_t head) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row % 8 == 0 && head % 8 == 0;
}

}  // namespace

int kv_check(const wcomp_kv4* c, const wcomp_kv4_seqs& s, int64_t T) {
  if (!c || s.B < 0 || s.width < 1 || T < 0 || (s.B && (!s.d_table || !s.d_lengths))) return WCOMP_EINVAL;
  if (!s.d_starts && T != s.B) return WCOMP_EINVAL;
  if (!natural(s.d_table) || !natural(s.d_lengths) || !natural(s.d_starts)) return WCOMP_EINVAL;
  if (int64_t(s.width) * kPage > (int64_t(1) << 30) || T >= (int64_t(1) << 31)) return WCOMP_EUNSUPPORTED;
  return WCOMP_OK;
}

int kv_seqs(const wcomp_kv4* c, const wcomp_kv4_seqs& s, KvSeqs* out) {
  if (!on_device(c)) return WCOMP_EINVAL;
  *out = {s.d_table, s.d_lengths, s.d_starts, s.B, s.width, uint32_t(c->pages), uint32_t(c->heads), nullptr};
  return work_error(c->device, &out->err);
}

}  // namespace wc

using namespace wc;

// Calls f with a kernel's dim and steps: as many as the cache's heads fill.
template <class F>
static void kv_rows_kernel(const wcomp_kv4* c, F f) {
  auto steps = [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    if (c->heads <= Items<D, 1>::kHeads) f(dim, std::integral_constant<int, 1>{});
    else f(dim, std::integral_constant<int, 2>{});
  };
  if (c->dim == 64) steps(std::integral_constant<int, 64>{});
  else if (c->dim == 128) steps(std::integral_constant<int, 128>{});
  else steps(std::integral_constant<int, 256>{});
}
// Units of rows x heads: how many share rows, and rows of a warp.
struct RowUnits {
  uint32_t rounds, span, grid;
};
template <int D, int STEPS>
static RowUnits row_units(const wcomp_kv4* c, int64_t T) {
  RowUnits r;
  r.rounds = uint32_t(cdiv(uint64_t(c->heads), Items<D, STEPS>::kHeads));
  r.span = 1;
  while (r.span < kMaxSpan && T * r.rounds >= int64_t(sm_count(c->device)) * 64 * r.span) r.span *= 2;
  r.grid = grid_of(int64_t(cdiv(cdiv(uint64_t(T), r.span) * r.rounds, kThreads / 32)), c->device);
  return r;
}

#define WCOMP_KV_DIM(dim, CALL)       \
  do {                                \
    if ((dim) == 64) CALL(64);        \
    else if ((dim) == 128) CALL(128); \
    else CALL(256);                   \
  } while (0)

extern "C" int wcomp_kv4_create(int64_t pages, int heads, int dim, void* stream, wcomp_kv4** out) {
  if (out) *out = nullptr;
  if (!out || pages < 1 || heads < 1 || dim < 1) return WCOMP_EINVAL;
  if ((dim != 64 && dim != 128 && dim != 256) || pages >= (int64_t(1) << 31) || heads >= (1 << 16) ||
      pages * heads >= (int64_t(1) << 31))
    return WCOMP_EUNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return map_cuda(cudaGetLastError());
  uint32_t* err = nullptr;
  const int st = work_error(dev, &err);
  if (st != WCOMP_OK) return st;
  wcomp_kv4* c = new (std::nothrow) wcomp_kv4;
  if (!c) return WCOMP_ENOMEM;
  c->pages = pages;
  c->heads = heads;
  c->dim = dim;
  c->device = dev;
  const uint64_t bytes = uint64_t(pages) * heads * 72 * dim;
  cudaError_t e = pool_alloc(reinterpret_cast<void**>(&c->d), bytes, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(c->d, 0, bytes, s);  // scales of 0
  if (e != cudaSuccess) {
    cudaGetLastError();
    wcomp_kv4_free(c, stream);
    return map_cuda(e);
  }
  *out = c;
  return WCOMP_OK;
}

extern "C" int wcomp_kv4_append(wcomp_kv4* c, const wcomp_kv4_seqs* seqs, const uint16_t* d_k, int64_t k_row,
                                int64_t k_head, const uint16_t* d_v, int64_t v_row, int64_t v_head, int64_t T,
                                void* stream) {
  if (!seqs || (T && (!d_k || !d_v)) || k_row < 0 || k_head < 0 || v_row < 0 || v_head < 0 || !natural(d_k) || !natural(d_v))
    return WCOMP_EINVAL;
  int st = kv_check(c, *seqs, T);
  if (st != WCOMP_OK) return st;
  KvSeqs s;
  if ((st = kv_seqs(c, *seqs, &s)) != WCOMP_OK) return st;
  if (T == 0 || s.B == 0) return WCOMP_OK;
  const Rows k{d_k, k_row, k_head, rows_vec(d_k, k_row, k_head)}, v{d_v, v_row, v_head, rows_vec(d_v, v_row, v_head)};
  kv_rows_kernel(c, [&](auto dim, auto steps) {
    constexpr int D = decltype(dim)::value, STEPS = decltype(steps)::value;
    const RowUnits r = row_units<D, STEPS>(c, T);
    kv4_append_kernel<D, STEPS><<<r.grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(s, c->d, k, v, T, r.rounds, r.span);
  });
  count_launches(1);
  return map_cuda(cudaGetLastError());
}

extern "C" int wcomp_kv4_read(const wcomp_kv4* c, const wcomp_kv4_seqs* seqs, uint16_t* d_k, uint16_t* d_v, int64_t T,
                              void* stream) {
  if (!seqs || (T && (!d_k || !d_v)) || !natural(d_k) || !natural(d_v)) return WCOMP_EINVAL;
  int st = kv_check(c, *seqs, T);
  if (st != WCOMP_OK) return st;
  KvSeqs s;
  if ((st = kv_seqs(c, *seqs, &s)) != WCOMP_OK) return st;
  if (T == 0 || s.B == 0) return WCOMP_OK;
  const int vec = rows_vec(d_k, 0, 0) && rows_vec(d_v, 0, 0);
  kv_rows_kernel(c, [&](auto dim, auto steps) {
    constexpr int D = decltype(dim)::value, STEPS = decltype(steps)::value;
    const RowUnits r = row_units<D, STEPS>(c, T);
    kv4_read_kernel<D, STEPS><<<r.grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(s, c->d, d_k, d_v, T, r.rounds, r.span, vec);
  });
  count_launches(1);
  return map_cuda(cudaGetLastError());
}

extern "C" int wcomp_kv4_evict(wcomp_kv4* c, const wcomp_kv4_evict_args* args, void* stream) {
  if (!c || !args) return WCOMP_EINVAL;
  const wcomp_kv4_evict_args& a = *args;
  if (a.B < 0 || a.keep < 1 || a.recent < 0 || a.recent > a.keep || a.width_out < 1 ||
      int64_t(a.width_out) * kPage < a.keep)
    return WCOMP_EINVAL;
  if (a.B && (!a.d_mass || !a.d_table_out || !a.d_lengths_out || !a.d_mass_out || a.d_mass == a.d_mass_out ||
              a.d_table == a.d_table_out || a.d_lengths == a.d_lengths_out))
    return WCOMP_EINVAL;
  if (!natural(a.d_mass) || !natural(a.d_table_out) || !natural(a.d_lengths_out) || !natural(a.d_mass_out) ||
      !natural(a.d_kept))
    return WCOMP_EINVAL;
  int st = kv_check(c, {a.d_table, a.d_lengths, nullptr, a.B, a.width}, a.B);
  if (st != WCOMP_OK) return st;
  if (int64_t(a.width_out) * kPage > (int64_t(1) << 30) || int64_t(a.B) * c->heads >= (int64_t(1) << 28))
    return WCOMP_EUNSUPPORTED;
  EvictArgs p{};
  if ((st = kv_seqs(c, {a.d_table, a.d_lengths, nullptr, a.B, a.width}, &p.s)) != WCOMP_OK) return st;
  if (a.B == 0) return WCOMP_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.mass = a.d_mass;
  p.mass_out = a.d_mass_out;
  p.table_out = a.d_table_out;
  p.lengths_out = a.d_lengths_out;
  p.cache = c->d;
  p.width_out = a.width_out;
  p.keep = a.keep;
  p.recent = a.recent;
  p.kept = a.d_kept;
  const int64_t units = int64_t(a.B) * c->heads;
  if (!p.kept) {
    const cudaError_t e = pool_alloc(reinterpret_cast<void**>(&p.kept), uint64_t(units) * a.keep * sizeof(int32_t), s);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return map_cuda(e);
    }
  }
  // blocks share a long sequence while that leaves each something and the GPU has room
  uint32_t team = 1;
  while (team < kMaxTeam && int64_t(a.width) * kPage > int64_t(team) * kChoose * (kHeld + kShared) &&
         units * team * 2 <= sm_count(c->device) * 4)
    team *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(uint32_t(units) * team);
  cfg.blockDim = dim3(kChoose);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = team;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = team > 1 ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_choose_kernel, p, team);
  if (e == cudaSuccess) {
    cfg.gridDim = dim3(grid_of(units * int64_t(cdiv(a.keep, kPage)), c->device));
    cfg.blockDim = dim3(kMove);
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
#define CALL(D) e = cudaLaunchKernelEx(&cfg, kv4_move_kernel<D>, p)
    WCOMP_KV_DIM(c->dim, CALL);
#undef CALL
    count_launches(2);
  }
  if (!a.d_kept) cudaFreeAsync(p.kept, s);
  return map_cuda(e);
}

extern "C" int wcomp_kv4_info(const wcomp_kv4* c, wcomp_kv4_info_t* info) {
  if (!c || !info) return WCOMP_EINVAL;
  info->pages = c->pages;
  info->heads = c->heads;
  info->dim = c->dim;
  info->bytes = uint64_t(c->pages) * c->heads * 72 * c->dim;
  return WCOMP_OK;
}

extern "C" void wcomp_kv4_free(wcomp_kv4* c, void* stream) {
  if (!c) return;
  if (c->d) cudaFreeAsync(c->d, static_cast<cudaStream_t>(stream));
  delete c;
}
