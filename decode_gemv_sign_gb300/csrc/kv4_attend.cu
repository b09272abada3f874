// Attention over the 4-bit key/value cache.
//
// One pass with the running maximum and sum of a softmax.  At a few query rows a
// cached head the cache is read once and little is done with it: moving it is the
// bound, and a block of 64 tokens and 128 columns (9216 bytes) leaves an SM some
// 390 cycles before the arithmetic falls behind the HBM.  So both products run on
// warp-level tensor-core MMAs with the codes as exact fp16 integers (tile.cuh):
//
//   S^T[token, row] = sum over groups of ks[token, group] * (Ck[token, group] . Q[row, group])
//     M = 16 tokens, N = 8 rows: a group's codes are two MMAs, whose sum enters S
//     under the group's scale; scores are as exact as fp32 sums of the products.
//   O^T[column, row] += Cv^T[column, token] * (vs[token, group] * P^T[token, row])
//     M = 16 columns of a group, N = 8 rows: the group's scale goes into P, which
//     one transposition of 8 x 8 turns from the accumulators' into the operand's order.
//
// A value row is read by token and transposed by a byte permutation of two
// tokens' words.  vs * P is rounded to fp16 under a power of two that follows the
// largest scale seen, which the sums O are kept under: one rounding of 2^-11, full
// precision for products down to 2^-28 of the largest scale's.  0 to 31 of its exponent
// are in the weights' own (ordinary values then cost nothing; their sum is freed of it),
// what is beyond that multiplies the scales, so that no weight is lost.  The softmax's
// reference is the running maximum rounded up to a whole power of two, so that
// going over to another scales exactly, by powers of two.
//
// Each warp takes an equal run of the call's (sequence, tile of rows, head, page)
// units through a ring of its own, a tile's beginning and end counted as one more.
// Where a tile's pages fall on several warps, a block joins its warps' parts in
// shared memory and a second kernel those of blocks, always in the same order.  A
// part's sums are kept under a power of two that brings its sum of weights l to 1/8: the
// sums of large values over many tokens are beyond fp32, their means are not.
// Lengths are on the device, so every block sums up the work of all sequences
// first.
//
// Where the tables leave a warp few pages even if a tile is given to one block or
// one cluster, that is done instead: one kernel without a workspace, the parts
// joined through the cluster's shared memory.  One sequence of 4097 tokens, 32 query
// and 8 cached heads: 12.5 us, cut anywhere 20.8.  A cluster that has all rows of a
// sequence and head adds their tokens' weights too: 16.4 us instead of 20.5 with the
// kernel that else does it.
#include <algorithm>
#include <cmath>

#include "cluster.cuh"
#include "kv4.cuh"

namespace wc {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttendArgs {
  KvSeqs s;
  const uint8_t* cache;
  const uint16_t* q;
  int64_t q_row, q_head;
  uint16_t* out;
  float* lse;   // or null
  float* mass;  // or null
  int64_t T;
  int q_heads, share, window;
  int q_vec, out_vec;  // q's rows are 16-byte, out 8-byte aligned
  float scale;
  // workspace
  float* lse2;       // [T, q_heads], in base 2, or null (with mass)
  float* scores;     // [B, heads, width, share, 64], in base 2, or null (with mass)
  float* part;       // [2 warps][rows][D]: sums times down_of(sum of weights)
  float2* part_ml;   // [2 warps][rows]: maximum (base 2) and sum
  uint32_t warps;    // of the attention kernel
};

// ---------------------------------------------------------------------------
// Units.
// ---------------------------------------------------------------------------
// u / d, by the short division where u has 32 bits.
__device__ __forceinline__ uint64_t quotient(uint64_t u, uint64_t d) {
  return (u | d) >> 32 ? u / d : uint32_t(u) / uint32_t(d);
}
struct Seq {
  int n, rows;     // tokens, and rows of the call
  int64_t first;   // first row
  int tiles;       // of R (row, head of the group) pairs
  int page0, pages;
};

// TILES: every tile of rows is work of its own; else a page is one unit for all of
// them.  A sequence with rows has at least one page, also where it has no token.  A
// tile and head has one unit before its pages: what it costs to begin and end.
// (Without it the warps of 16 sequences of 0 to 16384 tokens that had the short ones
// took twice as long as the others.)
template <int R, bool TILES>
__device__ __forceinline__ Seq load_seq(const AttendArgs& a, int b) {
  Seq q;
  q.n = kv_length(a.s, b);
  if (a.s.starts) {
    q.first = a.s.starts[b];
    const int64_t rows = a.s.starts[b + 1] - q.first;
    q.rows = int(rows < 0 ? 0 : rows > a.T ? a.T : rows);
  } else {
    q.first = b;
    q.rows = 1;
  }
  q.tiles = TILES ? (q.rows * a.share + R - 1) / R : q.rows ? 1 : 0;
  const int at = q.n - q.rows;  // position of the first row; at - window alone may leave 32 bits
  const int lo = a.window && at >= a.window ? at - a.window + 1 : 0;
  q.page0 = min(lo, max(q.n - 1, 0)) / kPage;
  q.pages = max(1, (q.n + kPage - 1) / kPage - q.page0);
  return q;
}
__device__ __forceinline__ uint64_t seq_units(const AttendArgs& a, const Seq& q) {
  return uint64_t(q.tiles) * a.s.heads * (uint64_t(q.pages) + 1);
}

// Units before the sequences of each thread's share, [threads + 1] in shared
// memory.
template <int THREADS, int R, bool TILES>
__device__ __forceinline__ void sum_units(const AttendArgs& a, uint64_t* s_before, uint64_t* s_warp) {
  const int per = (a.s.B + THREADS - 1) / THREADS;
  const int b0 = min(a.s.B, int(threadIdx.x) * per), b1 = min(a.s.B, b0 + per);
  uint64_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += seq_units(a, load_seq<R, TILES>(a, b));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t x = sum;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  uint64_t before = x - sum;
  for (int w = 0; w < warp; ++w) before += s_warp[w];
  s_before[threadIdx.x] = before;
  if (threadIdx.x == THREADS - 1) s_before[THREADS] = before + sum;
  __syncthreads();
}

// A place in the units' order: sequence, tile, head and page, pages fastest.  Kept
// in shared memory, one for a warp's sums and one for its copies, and moved on by
// lane 0: registers are what the products want.
template <int THREADS, int R, bool TILES>
struct Walk {
  int b, page, tile;  // page -1: the unit before the pages
  uint32_t head;
  Seq q;
  __device__ __forceinline__ void find(const AttendArgs& a, const uint64_t* s_before, uint64_t u) {
    int lo = 0, hi = THREADS;  // s_before[lo] <= u < s_before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_before[mid] <= u) lo = mid;
      else hi = mid;
    }
    b = lo * ((a.s.B + THREADS - 1) / THREADS);
    u -= s_before[lo];
    q = load_seq<R, TILES>(a, b);
    for (uint64_t w; u >= (w = seq_units(a, q));) {
      u -= w;
      q = load_seq<R, TILES>(a, ++b);
    }
    const uint64_t seg = quotient(u, uint32_t(q.pages) + 1);
    page = int(u - seg * (uint32_t(q.pages) + 1)) - 1;
    tile = int(quotient(seg, a.s.heads));
    head = uint32_t(seg - uint64_t(tile) * a.s.heads);
  }
  // The next unit, which there is.
  __device__ __forceinline__ void next(const AttendArgs& a) {
    if (++page < q.pages) return;
    page = -1;
    if (++head < a.s.heads) return;
    head = 0;
    if (++tile < q.tiles) return;
    tile = 0;
    do q = load_seq<R, TILES>(a, ++b);
    while (q.tiles == 0);
  }
};

// The units of warp w of W: first(w) .. first(w + 1).  With fewer units than warps
// every block has some.
struct Runs {
  uint64_t total;
  uint32_t W;
  __device__ __forceinline__ uint64_t first(uint32_t w) const { return quotient(total * w, W); }
  __device__ __forceinline__ uint32_t of(uint64_t unit) const { return uint32_t(quotient((unit + 1) * W - 1, total)); }
};

// A ring's stage: a block, or half of one.
template <int D, bool HALF>
struct KvSrc {
  static constexpr uint32_t kStage = HALF ? Kv<D>::kHalf : Kv<D>::kBlock;
  static constexpr bool kCopies = true;
  typedef const uint8_t* Cursor;
  static __device__ __forceinline__ void issue(Cursor& c, uint32_t st, uint32_t bar) { bulk_copy(st, c, kStage, bar); }
};

// The blocks of a warp's units through its ring, ahead of their use: a block a stage,
// their keys alone, or (VALUES) their keys and then their values in stages of halves.
template <int D, class RING, class WALK, bool VALUES = false>
struct Pages {
  WALK& it;
  uint64_t left = 0;      // units to come
  uint32_t run = 0;       // of which the next are the pages `id` of lanes from, from + 1, ...
  int from = 0, id = 0;
  int base = -1, in = -1; // lane l's id is that of page base + l of sequence `in`
  uint32_t there = 0;     // bit per slot: its page exists
  const uint8_t* head = nullptr;
  const uint8_t* values = nullptr;
  __device__ __forceinline__ Pages(WALK& walk, uint64_t count) : it(walk), left(count) {}
  __device__ __forceinline__ void enter(const AttendArgs& a, int lane) {
    __syncwarp();
    if (it.page < 0) {
      if (--left == 0) return;
      __syncwarp();
      if (lane == 0) it.page = 0;
      __syncwarp();
    }
    const int at = it.q.page0 + it.page;
    if (in != it.b || at < base || at >= base + 32) {
      in = it.b;
      base = at;
      id = at + lane < (it.q.n + kPage - 1) / kPage ? kv_page(a.s, it.b, at + lane) : -1;
    }
    from = at - base;
    run = uint32_t(min(left, uint64_t(min(32 - from, it.q.pages - it.page))));
    head = a.cache + uint64_t(it.head) * Kv<D>::kBlock;
    __syncwarp();
    if (lane == 0) {  // the unit after the run
      it.page += int(run) - 1;
      if (left > run) it.next(a);
    }
    __syncwarp();
  }
  // Copy the next unit's block to `slot`.  A page that does not exist is stood in for
  // by the cache's first, which nothing is read of.
  __device__ __forceinline__ void issue(const AttendArgs& a, RING& ring, uint32_t slot, int lane) {
    if (VALUES && values) {
      ring.refill(slot, values, lane);
      values = nullptr;
      return;
    }
    if (!left) return;
    if (!run) {
      enter(a, lane);
      if (!left) return;
    }
    const int page = __shfl_sync(0xffffffffu, id, from++);
    there = page >= 0 ? there | 1u << slot : there & ~(1u << slot);
    const uint8_t* p = head + uint64_t(uint32_t(max(page, 0))) * (a.s.heads * Kv<D>::kBlock);
    ring.refill(slot, p, lane);
    if (VALUES) values = p + Kv<D>::kHalf;
    --left;
    --run;
  }
};

// ---------------------------------------------------------------------------
// Products.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint2 lds_v2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = lds_u32(a);
  } else if constexpr (N == 2) {
    const uint2 v = lds_v2(a);
    w[0] = v.x; w[1] = v.y;
  } else {
    const uint4 v = lds_v4(a);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  }
}
// The words of a row at byte b: 16-byte pieces may be apart (Kv::at).
template <int D, int N>
__device__ __forceinline__ void row_words(uint32_t st, uint32_t t, uint32_t b, uint32_t (&w)[N]) {
  if constexpr (N <= 4) {
    lds_words<N>(st + Kv<D>::at(t, b), w);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = lds_v4(st + Kv<D>::at(t, b + 4 * i));
      w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
    }
  }
}

// 8 x 8 16-bit values across the warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A tile's rows: R = 8 NT (row, head of the group) pairs.  Lane (r, q) holds the
// operand's part of row 8 n + r and the state of the rows 8 n + 2 q + e.
template <int D, int NT>
struct Tile {
  static constexpr int G = Kv<D>::G;
  uint32_t b[NT][G][4];        // the pairs of columns (0, 4), (2, 6), (1, 5), (3, 7) of 32 g + 8 q ..
  float c[NT][2];              // what brings a score to base 2: |scale|, log2 e and the row's power of two
  int lo0, lo1, hi0, hi1;      // first and one past the last position seen: least and greatest of the tile's rows

  __device__ __forceinline__ void load(const AttendArgs& p, const Seq& s, int tile, int head, int lane) {
    const int r = lane >> 2, q = lane & 3;
    const int pairs = s.rows * p.share;
    const uint32_t flip = p.scale < 0.f ? 0x80000000u : 0u;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int x = tile * 8 * NT + 8 * n + r, tok = x / p.share;
      const int64_t i = s.first + tok;
      const bool ok = x < pairs && i >= 0 && i < p.T;
      const uint16_t* src = p.q + i * p.q_row + (head * p.share + x - tok * p.share) * p.q_head + 8 * q;
      uint32_t m = 0;
      uint32_t v[G][4];
#pragma unroll
      for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[g][k] = 0;
        if (ok) {
          if (p.q_vec) {
            const uint4 y = *reinterpret_cast<const uint4*>(src + 32 * g);
            v[g][0] = y.x; v[g][1] = y.y; v[g][2] = y.z; v[g][3] = y.w;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[g][k] = src[32 * g + 2 * k] | uint32_t(src[32 * g + 2 * k + 1]) << 16;
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) m = max(m, max(v[g][k] & 0x7FFFu, (v[g][k] >> 16) & 0x7FFFu));
      }
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = record_exponent(m << 16);
      const float up = __uint_as_float(__float_as_uint(power_of_two(e)) | flip);
      // above 0 also where the scale is 0 or underflows: -inf times it stays
      const float factor = fmaxf(fabsf(p.scale) * kLog2e * power_of_two(-e), 0x1p-126f);
#pragma unroll
      for (int g = 0; g < G; ++g) {  // columns 2 k, 2 k + 1 in v[g][k]
        b[n][g][0] = half2_bits(bf16_lo(v[g][0]) * up, bf16_lo(v[g][2]) * up);
        b[n][g][1] = half2_bits(bf16_lo(v[g][1]) * up, bf16_lo(v[g][3]) * up);
        b[n][g][2] = half2_bits(bf16_hi(v[g][0]) * up, bf16_hi(v[g][2]) * up);
        b[n][g][3] = half2_bits(bf16_hi(v[g][1]) * up, bf16_hi(v[g][3]) * up);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) c[n][k] = __shfl_sync(0xffffffffu, factor, 8 * q + 4 * k);
    }
    see(p, s, tile * 8 * NT / p.share, lo0, hi0);
    see(p, s, (min(pairs, (tile + 1) * 8 * NT) - 1) / p.share, lo1, hi1);
  }
  // What row `tok` of the sequence sees.
  static __device__ __forceinline__ void see(const AttendArgs& p, const Seq& s, int tok, int& lo, int& hi) {
    hi = max(0, s.n - s.rows + tok + 1);
    lo = p.window ? max(0, hi - p.window) : 0;
  }
  __device__ __forceinline__ bool sees_none(int page) const { return page * kPage >= hi1 || (page + 1) * kPage <= lo0; }
  __device__ __forceinline__ bool sees_all(int page) const { return page * kPage >= lo1 && (page + 1) * kPage <= hi0; }
  // Index of row 8 n + 2 q + k in lse (and, times D, in out), or -1; what it sees.
  static __device__ __forceinline__ int64_t row(const AttendArgs& p, const Seq& s, int tile, int head, int n, int k,
                                                int lane, int& lo, int& hi) {
    const int y = tile * 8 * NT + 8 * n + 2 * (lane & 3) + k, t = y / p.share;
    const int64_t j = s.first + t;
    see(p, s, t, lo, hi);
    if (y < s.rows * p.share && j >= 0 && j < p.T) return j * p.q_heads + head * p.share + (y - t * p.share);
    lo = hi = 0;
    return -1;
  }

  // Scores (before c) to their distances from `ref`, which they are rounded before: where a
  // score is 2^22 or more an fma would give the rounding as well, up to half a step above
  // ref, and a power of two beside ref would be lost.
  __device__ __forceinline__ void distances(const float (&ref)[NT][2], float (&z)[4][NT][4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float y = ref[n][k % 2];
          z[i][n][k] = __fsub_rn(__fmul_rn(z[i][n][k], c[n][k % 2]), y == -INFINITY ? 0.f : y);
        }
  }

  // Keep the scores of a page for kv4_weigh_kernel: the tile has all rows of the sequence.
  __device__ __forceinline__ void keep(const AttendArgs& p, int b, uint32_t head, int page, int lane,
                                       const float (&z)[4][NT][4]) const {
    const int r = lane >> 2, q = lane & 3;
    float* to = p.scores + ((uint64_t(b) * p.s.heads + head) * uint32_t(p.s.width) + uint32_t(page)) * uint32_t(p.share * kPage);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (8 * n + 2 * q + e < p.share) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            to[(8 * n + 2 * q + e) * kPage + 8 * k + r] = z[k / 2][n][e + 2 * (k % 2)] * c[n][e];
        }
  }

  // Scores (before c) of the keys at st: z[i][n][k + 2 h] of token 16 i + 8 h + r and row 8 n + 2 q + k.
  __device__ __forceinline__ void scores(uint32_t st, int lane, uint32_t magic, float (&z)[4][NT][4]) const {
    const uint32_t r = uint32_t(lane) >> 2, q = uint32_t(lane) & 3;
    uint32_t sc[G][4];  // word i: the scales of the tokens 16 i + r and 16 i + 8 + r
#pragma unroll
    for (int g = 0; g < G; ++g) lds_words<4>(st + Kv<D>::scale(r, g), sc[g]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[2][G];
      row_words<D, G>(st, 16 * i + r, q * G * 4, w[0]);
      row_words<D, G>(st, 16 * i + 8 + r, q * G * 4, w[1]);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint32_t x[4], y[4];
        q4_operand(w[0][g], magic, x);
        q4_operand(w[1][g], magic, y);
        const uint32_t a0[4] = {x[0], y[0], x[1], y[1]}, a1[4] = {x[2], y[2], x[3], y[3]};
        const float s0 = bf16_lo(sc[g][i]), s1 = bf16_hi(sc[g][i]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float d[4];
          mma_f16_first(d, a0, b[n][g][0], b[n][g][1]);
          mma_f16(d, a1, b[n][g][2], b[n][g][3]);
#pragma unroll
          for (int k = 0; k < 4; ++k) z[i][n][k] = g ? z[i][n][k] + (k < 2 ? s0 : s1) * d[k] : (k < 2 ? s0 : s1) * d[k];
        }
      }
    }
  }
};

// The power of two that brings a sum of weights to 1/8 .. 1/4, and back; one that is not
// 0 is at least 1/2.
__device__ __forceinline__ uint32_t exponent_of(float l) { return max(__float_as_uint(l) & 0x7F800000u, 126u << 23); }
__device__ __forceinline__ float down_of(float l) { return __uint_as_float((251u << 23) - exponent_of(l)); }
__device__ __forceinline__ float up_of(float l) { return __uint_as_float((3u << 23) + exponent_of(l)); }
constexpr float kFew = 16.f;  // parts of up to so many warps or blocks, whose largest l is `most`, are summed under down_of(most) / kFew

// Whether `ref`, of any row, is 2^22 or more from 0.
template <int NT>
__device__ __forceinline__ bool any_far(const float (&ref)[NT][2]) {
  bool far = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) far |= fabsf(ref[n][e]) >= 0x1p22f && fabsf(ref[n][e]) < INFINITY;
  return __any_sync(0xffffffffu, far);
}

// Multiply a page's scales of values by 2^d, in the warp's own stage: exact, but for those
// below 2^-140 of the largest.  Copies to the stage follow behind.
template <int D>
__device__ __forceinline__ void scale_scales(uint32_t at, int d, int lane) {
  const uint32_t f = __float_as_uint(power_of_two(d)) >> 16, f2 = f | f << 16;
  __syncwarp();
#pragma unroll
  for (uint32_t i = 0; i < Kv<D>::G; ++i) {
    uint32_t x = lds_u32(at + 4 * (32 * i + lane));
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(f2));
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 4 * (32 * i + lane)), "r"(x) : "memory");
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// Sums of a tile so far, and the softmax's state.
template <int D, int NT>
struct Sums {
  static constexpr int G = Kv<D>::G;
  static constexpr int kNoScale = 14 + 133;  // the least scale above 0 is 2^-133
  float m[NT][2], l[NT][2];  // reference (base 2, whole, or -inf) and, of the lane's tokens, sum
  float o[2 * G][NT][4];     // tile 2 g + i: column 32 g + 4 r + 2 i (+ 1: the last two) of the rows 2 q, 2 q + 1 (+ 8 n)
  int k;                     // o is under 2^k
  bool far;                  // a reference is far from 0 (Tile::distances)

  __device__ __forceinline__ void clear() {
    k = kNoScale;
    far = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = -INFINITY;
        l[n][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 2 * G; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][n][e] = 0.f;
    }
  }
  __device__ __forceinline__ void scale(int n, float f0, float f1) {
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) {
      o[i][n][0] *= f0;
      o[i][n][1] *= f1;
      o[i][n][2] *= f0;
      o[i][n][3] *= f1;
    }
  }

  // Add a page: scores z, values at st.  ALL: every row sees every token.
  template <bool ALL, class WALK>
  __device__ __forceinline__ void add(const AttendArgs& p, const WALK& at, const Tile<D, NT>& t, int page, uint32_t st,
                                      int lane, uint32_t magic, float (&z)[4][NT][4]) {
    const uint32_t r = uint32_t(lane) >> 2, q = uint32_t(lane) & 3;
    uint32_t seen[NT][2];  // bit 2 i + h: the token 16 i + 8 h + r
    if (!ALL) {
      const int from = page * kPage + int(r);
      auto below = [&](int end) {  // bits of the tokens before `end`
        const int k = (end - from + 7) >> 3;
        return k <= 0 ? 0u : k >= 8 ? 0xFFu : (1u << k) - 1u;
      };
      const bool alike = t.lo0 == t.lo1 && t.hi0 == t.hi1;  // all rows see the same
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          int lo = t.lo0, hi = t.hi0;
          if (!alike) Tile<D, NT>::row(p, at.q, at.tile, int(at.head), n, e, lane, lo, hi);
          seen[n][e] = below(hi) & ~below(lo);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (!(seen[n][e] >> k & 1)) z[k / 2][n][e + 2 * (k % 2)] = -INFINITY;
        }
    }
    bool more = false;
    float next[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(z[0][n][e], z[0][n][e + 2]);
#pragma unroll
        for (int i = 1; i < 4; ++i) x = fmaxf(x, fmaxf(z[i][n][e], z[i][n][e + 2]));
#pragma unroll
        for (int d = 4; d <= 16; d *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
        next[n][e] = fmaxf(m[n][e], ceilf(x * t.c[n][e]));
        more |= next[n][e] > m[n][e] || far;
      }
    if (__any_sync(0xffffffffu, more)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f[e] = next[n][e] > m[n][e] ? exp2_approx(m[n][e] - next[n][e]) : 1.f;
          m[n][e] = next[n][e];
          l[n][e] *= f[e];
        }
        scale(n, f[0], f[1]);
      }
      far = any_far<NT>(m);
      if (far) t.distances(m, z);
    }
    // the largest scale of a value that some row sees: G words a lane, 2 tokens each
    uint32_t top[G];
    if constexpr (G <= 4) {
      lds_words<G>(st + Kv<D>::kCodes + 4 * G * lane, top);
    } else {
#pragma unroll
      for (int i = 0; i < G; i += 4) {
        const uint4 v = lds_v4(st + Kv<D>::kCodes + 4 * (G * lane + i));
        top[i] = v.x; top[i + 1] = v.y; top[i + 2] = v.z; top[i + 3] = v.w;
      }
    }
    if (!ALL) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int e = 2 * ((G * lane + i) % 32);  // place of the first in its group (Kv::scale)
        const int at = page * kPage + (e >> 3) + 8 * (e & 7);
        if (at < t.lo0 || at >= t.hi1) top[i] &= 0xFFFF0000u;
        if (at + 8 < t.lo0 || at + 8 >= t.hi1) top[i] &= 0xFFFFu;
      }
    }
#pragma unroll
    for (int i = 1; i < G; ++i)  // a NaN loses against a number
      asm("max.bf16x2 %0, %0, %1;" : "+r"(top[0]) : "r"(top[i]));
    uint32_t hi = top[0] >> 16, lo = top[0] & 0xFFFFu;
    if (hi > 0x7F80u) hi = 0;
    if (lo > 0x7F80u) lo = 0;
    const uint32_t largest = __reduce_max_sync(0xffffffffu, max(hi, lo));
    int kw = k;  // of k, what is in the weights
    if (int(largest >> 7) + k > 14 + 127 || uint32_t(k) > 31u) {
      // 14 less the exponent of the largest, BF16's normal numbers or those below
      const int to = largest < 0x80u ? kNoScale - 31 + __clz(largest) : 14 + 127 - int(largest >> 7);
      if (largest && to < k) {
        const int d = max(to - k, -252);  // beyond it nothing is left either
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          scale(n, power_of_two(d / 2), power_of_two(d / 2));
          scale(n, power_of_two(d - d / 2), power_of_two(d - d / 2));
        }
        k = to;
      }
      kw = min(max(k, 0), 31);
      if (k != kw) scale_scales<D>(st + Kv<D>::kCodes, k - kw, lane);
    }
    uint64_t w2[4][NT][2];  // weights under 2^kw, a row's of the tokens 16 i + r and 16 i + 8 + r together
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float shift = far ? float(kw) : float(kw) - (m[n][e] == -INFINITY ? 0.f : m[n][e]);
        const float c = far ? 1.f : t.c[n][e];
        const uint64_t c2 = pair(c, c), shift2 = pair(shift, shift);
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t x = fma2(pair(z[i][n][e], z[i][n][e + 2]), c2, shift2);
          w2[i][n][e] = pair(exp2_approx(first(x)), exp2_approx(second(x)));
          sum = i ? add2(sum, w2[i][n][e]) : w2[i][n][e];
        }
        l[n][e] = __fmaf_rn(first(sum) + second(sum), power_of_two(-kw), l[n][e]);
      }
    uint32_t sc[G][4];
#pragma unroll
    for (int g = 0; g < G; ++g) lds_words<4>(st + Kv<D>::scale(r, g), sc[g]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4][G / 2];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        row_words<D, G / 2>(st, 16 * i + 8 * (e / 2) + 2 * q + e % 2, r * (G / 2) * 4, w[e]);
#pragma unroll
      for (int a = 0; a < G / 2; ++a) {
#pragma unroll
        for (int side = 0; side < 2; ++side) {  // groups 2 a and 2 a + 1
          const int g = 2 * a + side;
          const uint64_t s2 = pair(bf16_lo(sc[g][i]), bf16_hi(sc[g][i]));
          uint32_t b[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint64_t x0 = mul2(w2[i][n][0], s2), x1 = mul2(w2[i][n][1], s2);
            float x[4] = {first(x0), first(x1), second(x0), second(x1)};
            if (!ALL) {
#pragma unroll
              for (int e = 0; e < 4; ++e)  // also where the scale is NaN
                if (!(seen[n][e % 2] >> (2 * i + e / 2) & 1)) x[e] = 0.f;
            }
            b[n][0] = transpose8(half2_bits(x[0], x[1]));
            b[n][1] = transpose8(half2_bits(x[2], x[3]));
          }
          const uint32_t pick = side ? 0x7632 : 0x5410;
          uint32_t u[4], v[4];
          q4_operand(prmt(w[0][a], w[1][a], pick), magic, u);  // columns 0, 2, 1, 3 of two tokens
          q4_operand(prmt(w[2][a], w[3][a], pick), magic, v);
          const uint32_t a0[4] = {u[0], u[2], v[0], v[2]}, a1[4] = {u[1], u[3], v[1], v[3]};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16(o[2 * g][n], a0, b[n][0], b[n][1]);
            mma_f16(o[2 * g + 1][n], a1, b[n][0], b[n][1]);
          }
        }
      }
    }
  }
};

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// Four columns of a row of out.
__device__ __forceinline__ void store_out(const AttendArgs& a, int64_t at, const float (&x)[4]) {
  const uint32_t lo = bf16x2_bits(x[0], x[1]), hi = bf16x2_bits(x[2], x[3]);
  if (a.out_vec) {
    *reinterpret_cast<uint2*>(a.out + at) = make_uint2(lo, hi);
  } else {
    a.out[at] = uint16_t(lo);
    a.out[at + 1] = uint16_t(lo >> 16);
    a.out[at + 2] = uint16_t(hi);
    a.out[at + 3] = uint16_t(hi >> 16);
  }
}
__device__ __forceinline__ void store_lse(const AttendArgs& a, int64_t row, float m, float l) {
  const float y = m + log2f(l);  // -inf where nothing is seen
  if (a.lse) a.lse[row] = y * kLn2;
  if (a.lse2) a.lse2[row] = y;
}

// What a row of sequence b gets in place of 1 / its sum of weights where that is 0: 0 if it
// sees no token; NaN, for 0 / 0, if all scores are -inf.
__device__ __noinline__ float no_weight(const AttendArgs& a, int b, int lo, int hi) {
#pragma unroll 1
  for (int page = lo / kPage; page * kPage < hi; ++page)
    if (kv_page(a.s, b, page) >= 0) return NAN;
  return 0.f;
}

// What a tile's rows give to the tokens' weights: exp2(score - log-sum-exp), summed.
template <int D, int NT>
struct Weights {
  float lse[NT][2];  // base 2
  int lo[NT][2], hi[NT][2];
  bool far = false;
  // lse_of(index in lse, row of the tile)
  template <class F>
  __device__ __forceinline__ void load(const AttendArgs& a, const Seq& s, int tile, int head, int lane, F lse_of) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t row = Tile<D, NT>::row(a, s, tile, head, n, e, lane, lo[n][e], hi[n][e]);
        const float y = lse_of(row, 8 * n + 2 * (lane & 3) + e);
        lse[n][e] = row >= 0 ? y : INFINITY;  // a place without a row adds 0
      }
    far = any_far<NT>(lse);
  }
  // Add the scores z of a page to the sums of its tokens 8 k + r.
  __device__ __forceinline__ void add(const Tile<D, NT>& tile, int page, int lane, float (&z)[4][NT][4],
                                      float (&sum)[8]) const {
    const int r = lane >> 2;
    if (far) tile.distances(lse, z);
    const bool all = tile.sees_all(page);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float c = far ? 1.f : tile.c[n][e], from = far ? 0.f : lse[n][e];
        if (all) {
#pragma unroll
          for (int k = 0; k < 8; ++k) sum[k] += exp2_approx(__fmaf_rn(z[k / 2][n][e + 2 * (k % 2)], c, -from));
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (page * kPage + 8 * k + r >= lo[n][e] && page * kPage + 8 * k + r < hi[n][e])
              sum[k] += exp2_approx(__fmaf_rn(z[k / 2][n][e + 2 * (k % 2)], c, -from));
        }
      }
  }
};
// The sums of a page's tokens to mass.
__device__ __forceinline__ void add_mass(const AttendArgs& a, int b, uint32_t head, int n, int page, int lane,
                                         float (&sum)[8]) {
  // over the four lanes of a token: after each exchange a lane goes on with half of them
#pragma unroll
  for (int d = 4, bit = 1; d >= 2; d /= 2, bit *= 2) {
#pragma unroll
    for (int k = 0; k < d; ++k) {
      const float keep = (lane & bit) ? sum[k + d] : sum[k], give = (lane & bit) ? sum[k] : sum[k + d];
      sum[k] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
    }
  }
  const int pos = page * kPage + 8 * (4 * (lane & 1) + (lane & 2)) + (lane >> 2);
  float* mass = a.mass + (uint64_t(b) * a.s.heads + head) * (uint64_t(a.s.width) * kPage) + pos;
  if (pos < n) mass[0] += sum[0];
  if (pos + 8 < n) mass[8] += sum[1];
}

// Warps, and what a warp's ring holds: blocks, or halves of blocks (the weights'
// kernel, which reads keys alone, and where two blocks of eight warps are too much).
// The rings fill an SM's shared memory.  64 sequences of 8192 tokens, 8 cached heads,
// us by warps x blocks (h: halves), the shapes taken first:
//   128 columns,  8 rows: 12 x 2 127, 12 x 1 140, 16 x 1 137, 20 x 1 160, 10 x 2 167;
//                16 rows: 8 x 3 188, 12 x 2 257 (168 registers a thread spill);
//    64 columns,  8 rows: 16 x 3 78, 12 x 4 80;
//   256 columns,  8 rows: 8 x 3 h 247, 8 x 1 264, 6 x 2 307, 4 x 3 402.
template <int D, int NT>
struct Shape {
  static constexpr int kWarps = D == 64 ? (NT == 1 ? 16 : 12) : D == 128 ? (NT == 1 ? 12 : 8) : 8;
  static constexpr int kBlocks = D == 64 ? (NT == 1 ? 3 : 4) : D == 128 ? (NT == 1 ? 2 : 3) : 1;
  static constexpr int kHalves = D == 256 ? 3 : 2 * kBlocks;
  static constexpr bool kSplit = D == 256;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr uint32_t kSmem = kWarps * kHalves * (Kv<D>::kHalf + 8) + 128;
};

template <int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, 1) kv4_attend_kernel(const __grid_constant__ AttendArgs a) {
  constexpr bool kSplit = Shape<D, NT>::kSplit;
  constexpr int kThreads = Shape<D, NT>::kThreads, kWarps = Shape<D, NT>::kWarps, R = 8 * NT;
  constexpr int kDepth = kSplit ? Shape<D, NT>::kHalves : Shape<D, NT>::kBlocks;
  using Src = KvSrc<D, kSplit>;
  using W = Walk<kThreads, R, true>;
  __shared__ uint64_t s_before[kThreads + 1], s_warp[kWarps];
  __shared__ W s_at[kWarps][2];
  __shared__ uint64_t s_first[kWarps + 1];
  __shared__ int s_inner[kWarps];  // whether the warp's run begins and ends within one tile
  __shared__ float2 s_ml[kWarps][R];
  extern __shared__ __align__(128) uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t smem = smem_u32(smem_raw) + (-smem_u32(smem_raw) & 127u);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t magic = q4_magic();
  Ring<Src, kDepth> ring(smem + uint32_t(warp) * kDepth * Src::kStage,
                         smem + kWarps * kDepth * Src::kStage + uint32_t(warp) * kDepth * 8, a.s.err, lane);
  sum_units<kThreads, R, true>(a, s_before, s_warp);
  const Runs runs{s_before[kThreads], a.warps};
  const uint32_t me = blockIdx.x * kWarps + uint32_t(warp);
  if (threadIdx.x <= kWarps) s_first[threadIdx.x] = runs.first(blockIdx.x * kWarps + threadIdx.x);
  __syncthreads();
  uint64_t u = s_first[warp];
  const uint64_t end = s_first[warp + 1];
  W& at = s_at[warp][0];
  if (lane == 0 && u < end) {
    at.find(a, s_before, u);
    s_at[warp][1] = at;
  }
  if (lane == 0) s_inner[warp] = 0;
  __syncwarp();
  Pages<D, Ring<Src, kDepth>, W, kSplit> pages(s_at[warp][1], end - u);
#pragma unroll 1
  for (int i = 0; i < kDepth; ++i) pages.issue(a, ring, uint32_t(i), lane);
  Tile<D, NT> tile;
  Sums<D, NT> sums;
  const uint32_t q = uint32_t(lane) & 3, r = uint32_t(lane) >> 2;
  while (u < end) {
    // a tile's pages, or those of them that fall on this warp
    if (at.page < 0) {
      if (++u == end) break;
      __syncwarp();
      if (lane == 0) at.page = 0;
      __syncwarp();
    }
    const bool first = at.page == 0;
    int page = at.q.page0 + at.page;
    const int stop = int(min(int64_t(at.q.page0 + at.q.pages), int64_t(page) + int64_t(end - u)));
    const bool last = stop == at.q.page0 + at.q.pages, whole = first && last, inner = !first && !last;
    tile.load(a, at.q, at.tile, int(at.head), lane);
    sums.clear();
    u += uint64_t(stop - page);
#pragma unroll 1
    for (; page < stop; ++page) {
      ring.wait(lane);
      const bool look = (pages.there >> ring.slot & 1) && !tile.sees_none(page);
      float z[4][NT][4];
      if (look) {
        tile.scores(ring.stage(), lane, magic, z);
        if (a.scores) tile.keep(a, at.b, at.head, page, lane, z);
      }
      if (kSplit) {
        __syncwarp();
        pages.issue(a, ring, ring.slot, lane);
        ring.next();
        ring.wait(lane);
      }
      if (look) {
        const uint32_t values = ring.stage() + (kSplit ? 0 : Kv<D>::kHalf);
        if (tile.sees_all(page)) sums.template add<true>(a, at, tile, page, values, lane, magic, z);
        else sums.template add<false>(a, at, tile, page, values, lane, magic, z);
      }
      __syncwarp();
      pages.issue(a, ring, ring.slot, lane);
      ring.next();
    }
    const float back0 = power_of_two(-sums.k / 2), back1 = power_of_two(sums.k / 2 - sums.k);
    // an inner part goes to the warp's own stages, which nothing is copied to any more
    float* part = inner ? reinterpret_cast<float*>(smem_raw + (smem - smem_u32(smem_raw)) + warp * kDepth * Src::kStage)
                        : a.part + (uint64_t(2 * me + first) * R) * D;
    float2* ml = inner ? s_ml[warp] : a.part_ml + uint64_t(2 * me + first) * R;
    if (inner && lane == 0) s_inner[warp] = 1;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // row 8 n + 2 q + e
        float l = sums.l[n][e];
#pragma unroll
        for (int d = 4; d <= 16; d *= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
        int lo, hi;
        const int64_t row = Tile<D, NT>::row(a, at.q, at.tile, int(at.head), n, e, lane, lo, hi);
        if (row < 0) {
          if (inner && r == 0) ml[8 * n + 2 * q + e] = make_float2(-INFINITY, 0.f);
          continue;
        }
        if (r == 0) {
          if (whole) store_lse(a, row, sums.m[n][e], l);
          else ml[8 * n + 2 * q + e] = make_float2(sums.m[n][e], l);
        }
        const float f = back0 * (!whole ? down_of(l) : l == 0.f ? no_weight(a, at.b, lo, hi) : 1.f / l);
#pragma unroll
        for (int i = 0; i < Kv<D>::G; ++i) {
          float x[4] = {sums.o[2 * i][n][e], sums.o[2 * i][n][2 + e], sums.o[2 * i + 1][n][e], sums.o[2 * i + 1][n][2 + e]};
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = x[k] * f * back1;
          if (whole)
            store_out(a, row * D + 32 * i + 4 * r, x);
          else
            *reinterpret_cast<float4*>(part + (8 * n + 2 * q + e) * D + 32 * i + 4 * r) =
                make_float4(x[0], x[1], x[2], x[3]);
        }
      }
    }
    __syncwarp();
    if (lane == 0 && u < end) {
      at.page = at.q.pages - 1;
      at.next(a);
    }
    __syncwarp();
  }
  // Join the inner parts of neighbouring warps, which are one tile's: each of them takes
  // some rows; the result is the first one's.  (Unrolled, these loops cost the one over the
  // pages registers: 192 to 195 us with 16 rows of 128 columns, 64 sequences of 8192.)
  __syncthreads();
  if (!s_inner[warp]) return;
  auto same = [&](int w) {
    return s_inner[w] && s_at[w][0].b == at.b && s_at[w][0].tile == at.tile && s_at[w][0].head == at.head;
  };
  int w0 = warp, w1 = warp + 1;
  // warps without a unit lie between the others where units are few
  for (int w = warp - 1; w >= 0 && (same(w) || s_first[w] == s_first[w + 1]); --w)
    if (s_inner[w]) w0 = w;
  for (int w = warp + 1; w < kWarps && (same(w) || s_first[w] == s_first[w + 1]); ++w)
    if (s_inner[w]) w1 = w + 1;
  int parts = 0, mine = 0;
  for (int w = w0; w < w1; ++w) {
    if (w < warp) mine += s_inner[w];
    parts += s_inner[w];
  }
  const uint64_t out = uint64_t(2 * (blockIdx.x * kWarps + w0)) * R;
  constexpr int V = D / 32;
#pragma unroll 1
  for (int row = mine; row < R; row += parts) {
    float m = -INFINITY, most = 0.f, l = 0.f, o[V] = {};
#pragma unroll 1
    for (int w = w0; w < w1; ++w)
      if (s_inner[w]) {
        m = fmaxf(m, s_ml[w][row].x);
        most = fmaxf(most, s_ml[w][row].y);
      }
    const float from = m == -INFINITY ? 0.f : m, down = down_of(most) / kFew;
#pragma unroll 1
    for (int w = w0; w < w1; ++w) {
      if (!s_inner[w]) continue;
      const float2 ml = s_ml[w][row];
      const float e = exp2_approx(ml.x - from), f = e * up_of(ml.y) * down;
      l += e * ml.y;
      const float* x = reinterpret_cast<const float*>(smem_raw + (smem - smem_u32(smem_raw)) + w * kDepth * Src::kStage) +
                       row * D + lane;
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] += f * x[32 * k];
    }
    if (lane == 0) a.part_ml[out + row] = make_float2(m, l);
#pragma unroll
    for (int k = 0; k < V; ++k) a.part[(out + row) * D + lane + 32 * k] = o[k] * (down_of(l) * (up_of(most) * kFew));
  }
}

// The sequence and tile of a place in the order of tiles: sequence b has those from
// its first row's pairs / R + b on.  False where there is no tile.
template <int R>
__device__ __forceinline__ bool tile_at(const AttendArgs& a, int64_t place, int& b, int& tile, Seq& s) {
  if (a.s.starts) {
    auto first = [&](int i) { return int64_t(max(a.s.starts[i], 0)) * a.share / R + i; };
    int lo = 0, hi = a.s.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first(mid) <= place) lo = mid;
      else hi = mid;
    }
    b = lo;
    place -= first(b);
    if (place < 0 || place >= (int64_t(1) << 31)) return false;
    tile = int(place);
  } else {
    const int per = (a.share + R - 1) / R;
    b = int(place / per);
    tile = int(place % per);
  }
  s = load_seq<R, true>(a, b);
  return tile < s.tiles;
}

// Join the blocks' parts of a tile and head: one block.  They are those of the first
// and the last warp that have pages of it and, for every block between or around
// them, of its first warp with none but the tile's.  Where they are follows from the
// lengths alone and is worked out while the attention still runs; then every load of
// a thread is in flight at once.  (With places read from the workspace, after the
// attention's end, one sequence of 262143 tokens, 64 query and 8 cached heads, took 80 us, now 76.)
constexpr int kAtOnce = 8, kMaxParts = 256;
template <int D, int NT, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) kv4_join_kernel(const __grid_constant__ AttendArgs a, int64_t tiles) {
  constexpr int R = 8 * NT, K = Shape<D, NT>::kWarps, kItems = R * D / 4;
  constexpr int kGroups = THREADS / kItems;  // of threads that share a tile's parts
  static_assert(kItems * kGroups == THREADS, "an item a thread");
  __shared__ uint64_t s_before[THREADS + 1], s_warp[THREADS / 32];
  __shared__ int s_place[kMaxParts], s_count[THREADS / 32];
  __shared__ float4 s_o[kGroups][kItems];
  __shared__ float2 s_ml[kGroups][R];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  sum_units<THREADS, R, true>(a, s_before, s_warp);
  if (blockIdx.x == 0) kv_check_starts(a.s, a.T, threadIdx.x, THREADS);  // for the attention too, which still runs
  const Runs runs{s_before[THREADS], a.warps};
  bool waited = false;
  for (int64_t unit = blockIdx.x; unit < tiles * a.s.heads; unit += gridDim.x) {
    const uint32_t head = uint32_t(unit % a.s.heads);
    const int64_t place = unit / a.s.heads;
    int b, tile;
    Seq s;
    if (!tile_at<R>(a, place, b, tile, s)) continue;
    const int per = (a.s.B + THREADS - 1) / THREADS;
    uint64_t f0 = s_before[b / per] + (uint64_t(tile) * a.s.heads + head) * (uint32_t(s.pages) + 1) + 1;
    for (int i = b / per * per; i < b; ++i) f0 += seq_units(a, load_seq<R, true>(a, i));
    const uint64_t f1 = f0 + uint32_t(s.pages);
    const uint32_t w0 = runs.of(f0), w1 = runs.of(f1 - 1);
    if (w0 == w1 || w1 >= a.warps) continue;
    const uint32_t c0 = w0 / K, blocks = w1 / K - c0 + 1;
    int at = -1;
    if (threadIdx.x < blocks + 2) {
      const uint32_t p = threadIdx.x;
      at = int(p == 0 ? (2 * w0 + 1) * R : 2 * w1 * R);
      if (p > 1) {
        const uint32_t lo = max(w0 + 1, (c0 + p - 2) * K), w = runs.of(runs.first(lo));
        at = w < min(w1, (c0 + p - 1) * K) ? int(2 * w * R) : -1;
      }
    }
    const uint32_t some = __ballot_sync(0xffffffffu, at >= 0);
    __syncthreads();
    if (threadIdx.x % 32 == 0) s_count[threadIdx.x / 32] = __popc(some);
    __syncthreads();
    int before = 0, parts = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < int(threadIdx.x / 32)) before += s_count[w];
      parts += s_count[w];
    }
    if (at >= 0) s_place[before + __popc(some & ((1u << threadIdx.x % 32) - 1u))] = at;
    const int group = int(threadIdx.x) / kItems, item = int(threadIdx.x) % kItems;
    const int row = 4 * item / D, col = 4 * item % D;
    int lo, hi;
    const int64_t to = Tile<D, NT>::row(a, s, tile, int(head), row / 8, row % 2, row % 8 / 2, lo, hi);
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
    waited = true;
    __syncthreads();
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (to >= 0) {  // others have left nothing there
      for (int p0 = group; p0 < parts; p0 += kGroups * kAtOnce) {
        float2 ml[kAtOnce];
        float4 x[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const int p = p0 + k * kGroups;
          ml[k] = make_float2(-INFINITY, 0.f);
          x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (p < parts) {
            ml[k] = a.part_ml[s_place[p] + row];
            x[k] = *reinterpret_cast<const float4*>(a.part + int64_t(s_place[p] + row) * D + col);
          }
        }
        float next = m;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) next = fmaxf(next, ml[k].x);
        const float from = next == -INFINITY ? 0.f : next, before = exp2_approx(m - from), had = before * up_of(l);
        m = next;
        l *= before;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const float f = exp2_approx(ml[k].x - from);
          l += ml[k].y * f;
          ml[k].x = f * up_of(ml[k].y);
        }
        const float down = down_of(l);
        o = make_float4(o.x * (had * down), o.y * (had * down), o.z * (had * down), o.w * (had * down));
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const float f = ml[k].x * down;
          o.x += x[k].x * f;
          o.y += x[k].y * f;
          o.z += x[k].z * f;
          o.w += x[k].w * f;
        }
      }
    }
    if constexpr (kGroups > 1) {
      s_o[group][item] = o;
      if (col == 0) s_ml[group][row] = make_float2(m, l);
      __syncthreads();
      if (group == 0 && to >= 0) {
        for (int g = 1; g < kGroups; ++g) m = fmaxf(m, s_ml[g][row].x);
        const float from = m == -INFINITY ? 0.f : m;
        l = 0.f;
        for (int g = 0; g < kGroups; ++g) l += s_ml[g][row].y * exp2_approx(s_ml[g][row].x - from);
        o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int g = 0; g < kGroups; ++g) {
          const float2 ml = s_ml[g][row];
          const float4 x = s_o[g][item];
          const float f = exp2_approx(ml.x - from) * up_of(ml.y) * down_of(l);
          o = make_float4(o.x + x.x * f, o.y + x.y * f, o.z + x.z * f, o.w + x.w * f);
        }
      }
    }
    if (group == 0 && to >= 0) {
      const float f = l == 0.f ? no_weight(a, b, lo, hi) : up_of(l) / l;
      const float x[4] = {o.x * f, o.y * f, o.z * f, o.w * f};
      store_out(a, to * D + col, x);
      if (col == 0) store_lse(a, to, m, l);
    }
    __syncthreads();
  }
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A tile and head by one block, or by a cluster of up to 16: every warp takes every
// (blocks x warps)-th page.
template <int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, 1)
    kv4_attend_team_kernel(const __grid_constant__ AttendArgs a, uint32_t team, bool weigh) {
  constexpr int kWarps = Shape<D, NT>::kWarps, kDepth = Shape<D, NT>::kBlocks, R = 8 * NT, V = D / 32;
  using Src = KvSrc<D, false>;
  struct At {
    Seq q;
    int tile;
    uint32_t head;
  };
  __shared__ float2 s_ml[kWarps][R], s_joined[R];
  __shared__ float s_lse[R];  // base 2, of the rows that this block finishes
  extern __shared__ __align__(128) uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t smem = smem_u32(smem_raw) + (-smem_u32(smem_raw) & 127u);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t magic = q4_magic();
  const uint32_t rank = team > 1 ? cluster_rank() : 0;
  Ring<Src, kDepth> ring(smem + uint32_t(warp) * kDepth * Src::kStage,
                         smem + kWarps * kDepth * Src::kStage + uint32_t(warp) * kDepth * 8, a.s.err, lane);
  At at;
  int b;
  at.head = blockIdx.x / team % a.s.heads;
  // the same for all of a cluster
  if (!tile_at<R>(a, blockIdx.x / team / a.s.heads, b, at.tile, at.q)) {
    if (blockIdx.x == 0) kv_check_starts(a.s, a.T, threadIdx.x, 32 * kWarps);
    return;
  }
  // a warp's pages in the sequence: first + k * stride; the ids of 32 of them at a time
  const int first = int(rank * kWarps) + warp, stride = int(team * kWarps);
  const int count = max(0, (at.q.pages - first + stride - 1) / stride), pages = (at.q.n + kPage - 1) / kPage;
  const uint8_t* const head = a.cache + uint64_t(at.head) * Kv<D>::kBlock;
  int id = -1, ahead = 0;
  uint32_t there = 0;
  auto issue = [&](uint32_t slot) {
    if (ahead == count) return;
    if (ahead % 32 == 0) {
      const int page = at.q.page0 + first + (ahead + lane) * stride;
      id = ahead + lane < count && page < pages ? kv_page(a.s, b, page) : -1;
    }
    const int page = __shfl_sync(0xffffffffu, id, ahead % 32);
    there = page >= 0 ? there | 1u << slot : there & ~(1u << slot);
    const uint8_t* p = head + uint64_t(uint32_t(max(page, 0))) * (a.s.heads * Kv<D>::kBlock);
    ring.refill(slot, p, lane);
    ++ahead;
  };
#pragma unroll 1
  for (int i = 0; i < kDepth; ++i) issue(uint32_t(i));
  Tile<D, NT> tile;
  Sums<D, NT> sums;
  tile.load(a, at.q, at.tile, int(at.head), lane);
  sums.clear();
#pragma unroll 1
  for (int k = 0; k < count; ++k) {
    const int page = at.q.page0 + first + k * stride;
    ring.wait(lane);
    if ((there >> ring.slot & 1) && !tile.sees_none(page)) {
      float z[4][NT][4];
      tile.scores(ring.stage(), lane, magic, z);
      if (tile.sees_all(page)) sums.template add<true>(a, at, tile, page, ring.stage() + Kv<D>::kHalf, lane, magic, z);
      else sums.template add<false>(a, at, tile, page, ring.stage() + Kv<D>::kHalf, lane, magic, z);
    }
    __syncwarp();
    issue(ring.slot);
    ring.next();
  }
  // The weights of its pages, once the rows' log-sum-exps are known (row's by lse_of); the
  // stages' stores and loads are behind a barrier.
  auto weigh_pages = [&](auto lse_of) {
    Weights<D, NT> weights;
    weights.load(a, at.q, at.tile, int(at.head), lane, [&](int64_t, int row) { return lse_of(row); });
    ahead = 0;
#pragma unroll 1
    for (uint32_t i = 0, slot = ring.slot; i < kDepth; ++i, slot = slot + 1 == kDepth ? 0 : slot + 1) issue(slot);
#pragma unroll 1
    for (int k = 0; k < count; ++k) {
      const int page = at.q.page0 + first + k * stride;
      ring.wait(lane);
      if ((there >> ring.slot & 1) && !tile.sees_none(page)) {
        float z[4][NT][4], sum[8] = {};
        tile.scores(ring.stage(), lane, magic, z);
        weights.add(tile, page, lane, z, sum);
        add_mass(a, b, at.head, at.q.n, page, lane, sum);
      }
      __syncwarp();
      issue(ring.slot);
      ring.next();
    }
  };
  // the warp's sums to its own stages
  const uint32_t q = uint32_t(lane) & 3, r = uint32_t(lane) >> 2;
  float* const stages = reinterpret_cast<float*>(smem_raw + (smem - smem_u32(smem_raw)));
  constexpr int kPart = kDepth * int(Src::kStage) / 4;
  const float back0 = power_of_two(-sums.k / 2), back1 = power_of_two(sums.k / 2 - sums.k);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = sums.l[n][e];
#pragma unroll
      for (int d = 4; d <= 16; d *= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
      const int row = 8 * n + 2 * int(q) + e;
      if (r == 0) s_ml[warp][row] = make_float2(sums.m[n][e], l);
      const float f = back0 * down_of(l);
#pragma unroll
      for (int i = 0; i < Kv<D>::G; ++i)
        *reinterpret_cast<float4*>(stages + warp * kPart + row * D + 32 * i + 4 * r) =
            make_float4(sums.o[2 * i][n][e] * f * back1, sums.o[2 * i][n][2 + e] * f * back1,
                        sums.o[2 * i + 1][n][e] * f * back1, sums.o[2 * i + 1][n][2 + e] * f * back1);
    }
  __syncthreads();
  // join the warps: each takes some rows
  const int parts = min(kWarps, max(0, at.q.pages - int(rank * kWarps)));
  constexpr int kRows = (R + kWarps - 1) / kWarps;
  float o[kRows][V], up[kRows];  // o is under 1 / up
  float2 ml[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int row = warp + j * kWarps;
    if (row >= R) break;
    float m = -INFINITY, most = 0.f, l = 0.f;
    for (int w = 0; w < parts; ++w) {
      m = fmaxf(m, s_ml[w][row].x);
      most = fmaxf(most, s_ml[w][row].y);
    }
    const float from = m == -INFINITY ? 0.f : m, down = down_of(most) / kFew;
#pragma unroll
    for (int k = 0; k < V; ++k) o[j][k] = 0.f;
#pragma unroll 4
    for (int w = 0; w < parts; ++w) {
      const float2 x = s_ml[w][row];
      const float e = exp2_approx(x.x - from), f = e * up_of(x.y) * down;
      l += e * x.y;
#pragma unroll
      for (int k = 0; k < V; ++k) o[j][k] += f * stages[w * kPart + row * D + lane + 32 * k];
    }
    ml[j] = make_float2(m, l);
    up[j] = up_of(most) * kFew;
  }
  auto finish = [&](int row, float m, float l, float up, const float (&x)[V]) {  // x under 1 / up
    int lo, hi;
    const int64_t to = Tile<D, NT>::row(a, at.q, at.tile, int(at.head), row / 8, row % 2, row % 8 / 2, lo, hi);
    if (to < 0) return;
    const float f = l == 0.f ? no_weight(a, b, lo, hi) : up / l;
#pragma unroll
    for (int k = 0; k < V; ++k) a.out[to * D + lane + 32 * k] = uint16_t(bf16x2_bits(x[k] * f, 0.f));
    if (lane == 0) {
      store_lse(a, to, m, l);
      s_lse[row] = m + log2f(l);
    }
  };
  if (team == 1) {
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      if (warp + j * kWarps < R) finish(warp + j * kWarps, ml[j].x, ml[j].y, up[j], o[j]);
    if (blockIdx.x == 0) kv_check_starts(a.s, a.T, threadIdx.x, 32 * kWarps);
    if (!weigh) return;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // copies follow stores to the stages
    __syncthreads();
    weigh_pages([&](int row) { return s_lse[row]; });
    return;
  }
  __syncthreads();  // the parts have been read
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int row = warp + j * kWarps;
    if (row >= R) break;
    if (lane == 0) s_joined[row] = ml[j];
    const float f = down_of(ml[j].y) * up[j];
#pragma unroll
    for (int k = 0; k < V; ++k) stages[row * D + lane + 32 * k] = o[j][k] * f;
  }
  cluster_sync();
  // join the blocks: a row a warp of all of them
  for (int row = int(rank) + int(team) * warp; row < R; row += int(team) * kWarps) {
    const float2 mine = lane < team ? make_float2(cluster_lds(smem_u32(&s_joined[row].x), lane),
                                                  cluster_lds(smem_u32(&s_joined[row].y), lane))
                                    : make_float2(-INFINITY, 0.f);
    float m = mine.x;
#pragma unroll
    for (int d = 16; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mine.y)));
    const float f = exp2_approx(mine.x - (m == -INFINITY ? 0.f : m)), down = down_of(most) / kFew;
    const float to = f * up_of(mine.y) * down;
    float l = 0.f, x[V] = {};
#pragma unroll 4
    for (uint32_t w = 0; w < team; ++w) {
      const float g = __shfl_sync(0xffffffffu, to, w);
      l += __shfl_sync(0xffffffffu, f * mine.y, w);
#pragma unroll
      for (int k = 0; k < V; ++k) x[k] += g * cluster_lds(smem + 4 * uint32_t(row * D + lane + 32 * k), w);
    }
    finish(row, m, l, up_of(most) * kFew, x);
  }
  if (weigh) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (blockIdx.x == 0) kv_check_starts(a.s, a.T, threadIdx.x, 32 * kWarps);
  cluster_sync();  // a block's shared memory stays while others read it
  if (!weigh) return;
  weigh_pages([&](int row) { return cluster_lds(smem_u32(&s_lse[row]), uint32_t(row) % team); });
  cluster_sync();
}

// The weight of every token: the scores again, from the keys alone, against the
// rows' log-sum-exps.
template <int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, 1) kv4_mass_kernel(const __grid_constant__ AttendArgs a) {
  constexpr int kThreads = Shape<D, NT>::kThreads, kWarps = Shape<D, NT>::kWarps, kDepth = Shape<D, NT>::kHalves,
                R = 8 * NT;
  using Src = KvSrc<D, true>;
  using W = Walk<kThreads, R, false>;
  __shared__ uint64_t s_before[kThreads + 1], s_warp[kWarps];
  __shared__ W s_at[kWarps][2];
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const uint32_t smem = smem_u32(smem_raw) + (-smem_u32(smem_raw) & 127u);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t magic = q4_magic();
  Ring<Src, kDepth> ring(smem + uint32_t(warp) * kDepth * Src::kStage,
                         smem + kWarps * kDepth * Src::kStage + uint32_t(warp) * kDepth * 8, a.s.err, lane);
  sum_units<kThreads, R, false>(a, s_before, s_warp);
  const Runs runs{s_before[kThreads], a.warps};
  uint64_t u = runs.first(blockIdx.x * kWarps + uint32_t(warp));
  const uint64_t end = runs.first(blockIdx.x * kWarps + uint32_t(warp) + 1);
  W& at = s_at[warp][0];
  if (lane == 0 && u < end) {
    at.find(a, s_before, u);
    s_at[warp][1] = at;
  }
  __syncwarp();
  Pages<D, Ring<Src, kDepth>, W> pages(s_at[warp][1], end - u);
#pragma unroll 1
  for (int i = 0; i < kDepth; ++i) pages.issue(a, ring, uint32_t(i), lane);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the log-sum-exps are there
  Tile<D, NT> tile;
  Weights<D, NT> weights;
  int b = -1, held = 0;
  uint32_t head = 0;  // what the tile holds
  for (; u < end; ++u) {
    if (at.page < 0) {
      __syncwarp();
      if (lane == 0) at.page = 0;
      __syncwarp();
      continue;
    }
    ring.wait(lane);
    const int page = at.q.page0 + at.page;
    if (pages.there >> ring.slot & 1) {
      float sum[8] = {};  // of the tokens 8 k + r
      const int tiles = (at.q.rows * a.share + R - 1) / R;
      for (int t = 0; t < tiles; ++t) {
        if (b != at.b || head != at.head || held != t) {
          b = at.b;
          head = at.head;
          held = t;
          tile.load(a, at.q, t, int(head), lane);
          weights.load(a, at.q, t, int(head), lane, [&](int64_t row, int) { return row >= 0 ? a.lse2[row] : 0.f; });
        }
        if (tile.sees_none(page)) continue;
        float z[4][NT][4];
        tile.scores(ring.stage(), lane, magic, z);
        weights.add(tile, page, lane, z, sum);
      }
      add_mass(a, at.b, at.head, at.q.n, page, lane, sum);
    }
    __syncwarp();
    pages.issue(a, ring, ring.slot, lane);
    ring.next();
    if (lane == 0 && u + 1 < end) at.next(a);
    __syncwarp();
  }
}

// The weight of every token from the scores that the attention has kept: for sequences
// of one row.  16 sequences of 16384 tokens, 128 columns, 4 query rows a cached head: the
// stores take 4 us of the attention's time and this 18, the keys again 54; 8 rows 32 and
// 55 (by columns and rows: at the launch).
constexpr int kWeigh = 512, kPagesAtOnce = 4;
__global__ void __launch_bounds__(kWeigh, 3) kv4_weigh_kernel(const __grid_constant__ AttendArgs a) {
  constexpr int kWarps = kWeigh / 32;
  using W = Walk<kWeigh, 8, false>;
  __shared__ uint64_t s_before[kWeigh + 1], s_warp[kWarps];
  __shared__ W s_at[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  sum_units<kWeigh, 8, false>(a, s_before, s_warp);
  const Runs runs{s_before[kWeigh], gridDim.x * kWarps};
  uint64_t u = runs.first(blockIdx.x * kWarps + uint32_t(warp));
  const uint64_t end = runs.first(blockIdx.x * kWarps + uint32_t(warp) + 1);
  W& at = s_at[warp];
  if (lane == 0 && u < end) at.find(a, s_before, u);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // scores and log-sum-exps are there
  __syncwarp();
  while (u < end) {
    if (at.page < 0) {
      if (++u == end) break;
      __syncwarp();
      if (lane == 0) at.page = 0;
      __syncwarp();
    }
    const int n = at.q.n, lo = a.window ? n - a.window : 0;
    const int from = at.q.page0 + at.page, stop = int(min(int64_t(at.q.page0 + at.q.pages), int64_t(from) + int64_t(end - u)));
    u += uint64_t(stop - from);
    const uint64_t first = (uint64_t(at.b) * a.s.heads + at.head) * uint32_t(a.s.width);  // of the sequence and head's pages
    const float lse = lane < a.share ? a.lse2[int64_t(at.b) * a.q_heads + at.head * uint32_t(a.share) + lane] : 0.f;
    for (int base = from; base < stop; base += 32) {
      const bool there = base + lane < stop && (base + lane) * kPage < n && kv_page(a.s, at.b, base + lane) >= 0;
      const uint32_t some = __ballot_sync(0xffffffffu, there);
      for (int j0 = 0; j0 < 32; j0 += kPagesAtOnce) {
        if (!(some >> j0 & ((1u << kPagesAtOnce) - 1u))) continue;
        const float2* x = reinterpret_cast<const float2*>(a.scores + (first + uint32_t(base + j0)) * uint32_t(a.share * kPage)) + lane;
        float2 sum[kPagesAtOnce] = {};
#pragma unroll 2
        for (int row = 0; row < a.share; ++row) {
          const float y = __shfl_sync(0xffffffffu, lse, row);
#pragma unroll
          for (int j = 0; j < kPagesAtOnce; ++j)
            if (some >> (j0 + j) & 1) {
              const float2 z = x[(j * a.share + row) * (kPage / 2)];
              sum[j].x += exp2_approx(z.x - y);
              sum[j].y += exp2_approx(z.y - y);
            }
        }
#pragma unroll
        for (int j = 0; j < kPagesAtOnce; ++j)
          if (some >> (j0 + j) & 1) {
            const int pos = (base + j0 + j) * kPage + 2 * lane;
            float* mass = a.mass + first * kPage + pos;
            if (pos >= lo && pos < n) mass[0] += sum[j].x;
            if (pos + 1 >= lo && pos + 1 < n) mass[1] += sum[j].y;
          }
      }
    }
    __syncwarp();
    if (lane == 0 && u < end) {
      at.page = at.q.pages - 1;
      at.next(a);
    }
    __syncwarp();
  }
}

template <class K, class... ARGS>
cudaError_t launch(K kernel, uint32_t grid, int threads, uint32_t smem, bool dependent, uint32_t cluster,
                   cudaStream_t s, const ARGS&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(uint32_t(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (dependent) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Once a device: the kernels' shared memory and clusters of 16 allowed; how many
// clusters of 1 << i blocks fit the GPU at a time: less than its SMs / 2^i where a
// group of SMs has some left over.  (2 sequences of 512 tokens, 64 query and 8 cached
// heads, in 16 clusters of 8, which do not fit at once: 18.4 us; in clusters of 4: 10.3.)
struct Clusters {
  bool known;
  int fit[5];
};
template <int D, int NT>
cudaError_t prepare(int dev, Clusters* out) {
  static std::mutex mu;
  static Clusters all[64];
  std::lock_guard<std::mutex> g(mu);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  Clusters& c = all[dev];
  if (!c.known) {
    constexpr int smem = int(Shape<D, NT>::kSmem);
    const auto limit = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(kv4_attend_kernel<D, NT>, limit, smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kv4_mass_kernel<D, NT>, limit, smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kv4_attend_team_kernel<D, NT>, limit, smem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kv4_attend_team_kernel<D, NT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    for (int i = 0; i < 5; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(1u << i);
      cfg.blockDim = dim3(uint32_t(Shape<D, NT>::kThreads));
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = 1u << i;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&c.fit[i], kv4_attend_team_kernel<D, NT>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        c.fit[i] = 0;
      }
    }
    c.known = true;
  }
  *out = c;
  return cudaSuccess;
}

// Blocks to a tile and head, or 0 where the units are cut anywhere: the largest
// cluster that all of them have room for at once, if its warps get at most four
// pages each by the table.  8 sequences of 6144 tokens, 64 query and 8 cached heads:
// 20.5 us by two blocks a tile and head, 28.8 cut anywhere; with all but the first an
// eighth as long 20.5 and 20.7.  At eight pages a warp (8 x 12288) the first are 34.8
// and 41.0, the second 30.8 and 24.6.
template <int D, int NT>
uint32_t team_of(const AttendArgs& a, int64_t segments, uint32_t sms, const Clusters& c) {
  if (segments > sms) return 0;
  uint32_t team = 1;
  for (int i = 1; i < 5 && segments << i <= sms && segments <= c.fit[i]; ++i) team = 1u << i;
  const int64_t pages = a.window ? std::min<int64_t>(a.s.width, (int64_t(a.window) + a.T) / kPage + 2) : a.s.width;
  return pages <= int64_t(4) * team * Shape<D, NT>::kWarps ? team : 0;
}

constexpr uint64_t kMostScores = uint64_t(256) << 20;

template <int D, int NT>
int attend(AttendArgs& a, int dev, cudaStream_t s) {
  constexpr int kThreads = Shape<D, NT>::kThreads;
  constexpr uint32_t smem = Shape<D, NT>::kSmem;
  const uint32_t sms = uint32_t(std::min(sm_count(dev), kMaxParts - 2));  // a part a block, and two
  Clusters clusters;
  cudaError_t e = prepare<D, NT>(dev, &clusters);
  if (e != cudaSuccess) return map_cuda(e);
  // places for the tiles of all sequences (tile_at)
  const int64_t tiles = a.s.starts ? a.T * a.share / (8 * NT) + a.s.B + 1
                                   : int64_t(a.s.B) * int64_t(cdiv(uint64_t(a.share), 8 * NT));
  const uint32_t team = team_of<D, NT>(a, tiles * a.s.heads, sms, clusters);
  a.warps = sms * Shape<D, NT>::kWarps;
  auto up = [](uint64_t x) { return (x + 255) & ~uint64_t(255); };
  const uint64_t slots = team ? 0 : uint64_t(2) * a.warps * 8 * NT;
  // where a cluster has all rows of a sequence and head it weighs the tokens too
  const bool weigh = a.mass && team && !a.s.starts && a.share <= 8 * NT;
  // Scores are kept rather than computed again where each sequence has one tile of them,
  // they are not too many, and they are no more than the keys are worth.  16 sequences of
  // 16384 tokens, 8 cached heads, the whole call kept / again: 64 columns, 1 query row a cached
  // head 63 / 88 us, 8 80 / 88, 9 108 / 116, 12 118 / 116, 16 130 / 117; 128 columns, 1 85 / 121,
  // 8 103 / 124, 16 165 / 180; 256 columns, 1 148 / 215, 8 167 / 218.
  const uint64_t scores = uint64_t(a.s.B) * a.s.heads * uint64_t(a.s.width) * uint64_t(a.share) * (kPage * 4);
  const bool kept =
      a.mass && !team && !a.s.starts && a.share <= 8 * NT && a.share * 6 <= D && scores <= kMostScores;
  const uint64_t b_lse = a.mass && !weigh ? up(uint64_t(a.T) * a.q_heads * 4) : 0, b_ml = up(slots * 8), b_part = slots * D * 4,
                 b_scores = kept ? scores : 0;
  uint8_t* ws = nullptr;
  if (b_lse + b_ml + b_part + b_scores) {
    e = pool_alloc(reinterpret_cast<void**>(&ws), b_lse + b_ml + b_part + b_scores, s);
    if (e != cudaSuccess) return map_cuda(e);
  }
  a.lse2 = a.mass && !weigh ? reinterpret_cast<float*>(ws) : nullptr;
  a.part_ml = reinterpret_cast<float2*>(ws + b_lse);
  a.part = reinterpret_cast<float*>(ws + b_lse + b_ml);
  a.scores = kept ? reinterpret_cast<float*>(ws + b_lse + b_ml + b_part) : nullptr;
  if (team) {
    e = launch(kv4_attend_team_kernel<D, NT>, uint32_t(tiles * a.s.heads) * team, kThreads, smem, false, team, s, a, team, weigh);
  } else {
    e = launch(kv4_attend_kernel<D, NT>, sms, kThreads, smem, false, 1, s, a);
    // few tiles have many parts: 1024 threads share them; many have two or three
    constexpr int kSmall = 8 * NT * D / 4 < 256 ? 256 : 8 * NT * D / 4;
    const int64_t joins = tiles * a.s.heads;
    if (e == cudaSuccess)
      e = joins <= sms ? launch(kv4_join_kernel<D, NT, 1024>, uint32_t(joins), 1024, 0, true, 1, s, a, tiles)
                       : launch(kv4_join_kernel<D, NT, kSmall>, uint32_t(std::min<int64_t>(joins, int64_t(sms) * 4)), kSmall,
                                0, true, 1, s, a, tiles);
  }
  if (e == cudaSuccess && kept) e = launch(kv4_weigh_kernel, sms * 3, kWeigh, 0, true, 1, s, a);
  else if (e == cudaSuccess && a.mass && !weigh) e = launch(kv4_mass_kernel<D, NT>, sms, kThreads, smem, true, 1, s, a);
  if (ws) cudaFreeAsync(ws, s);
  return map_cuda(e);
}

}  // namespace

WCOMP_DEBUG_HOOKS(debug_hooks_kv4)
}  // namespace wc

using namespace wc;

extern "C" int wcomp_kv4_attend(const wcomp_kv4* c, const wcomp_kv4_attend_args* args, void* stream) {
  if (!c || !args) return WCOMP_EINVAL;
  const wcomp_kv4_attend_args& a = *args;
  int st = kv_check(c, a.s, a.T);
  if (st != WCOMP_OK) return st;
  if (a.q_heads < 1 || a.q_heads % c->heads || a.window < 0 || !std::isfinite(a.scale) || a.q_row < 0 || a.q_head < 0 ||
      (a.T && (!a.d_q || !a.d_out || a.d_out == a.d_q)) || !natural(a.d_q) || !natural(a.d_out) || !natural(a.d_lse) ||
      !natural(a.d_mass))
    return WCOMP_EINVAL;
  if (a.T * a.q_heads >= (int64_t(1) << 31)) return WCOMP_EUNSUPPORTED;
  AttendArgs p{};
  if ((st = kv_seqs(c, a.s, &p.s)) != WCOMP_OK) return st;
  if (a.T == 0 || a.s.B == 0) return WCOMP_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.cache = c->d;
  p.q = a.d_q;
  p.q_row = a.q_row;
  p.q_head = a.q_head;
  p.q_vec = reinterpret_cast<uintptr_t>(a.d_q) % 16 == 0 && a.q_row % 8 == 0 && a.q_head % 8 == 0;
  p.out = a.d_out;
  p.out_vec = reinterpret_cast<uintptr_t>(a.d_out) % 8 == 0;
  p.lse = a.d_lse;
  p.mass = a.d_mass;
  p.T = a.T;
  p.q_heads = a.q_heads;
  p.share = a.q_heads / c->heads;
  p.window = a.window;
  p.scale = a.scale;
  // Tiles of 8 where sequences have no more (rows, heads of a group) on the average, else of
  // 16, which read a page once: 64 x 8192 tokens, 128 columns, 16 of each sequence 190 us,
  // in two tiles of 8 232; 8 of each 131, in half a tile of 16 187; 64 of every eighth
  // sequence, which the average takes for 8, 111 and 125.  With 256 columns the registers
  // do not hold 16.
  const bool one = p.share <= 8 && a.T * p.share <= int64_t(8) * a.s.B;
  if (c->dim == 64) return one ? attend<64, 1>(p, c->device, s) : attend<64, 2>(p, c->device, s);
  if (c->dim == 128) return one ? attend<128, 1>(p, c->device, s) : attend<128, 2>(p, c->device, s);
  return attend<256, 1>(p, c->device, s);
}
