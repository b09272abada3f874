// Log probabilities, entropy and top alternatives from logits.
//
// A row is read once, by a block of 256 threads or, where there are few rows, by a
// cluster of blocks that share it; what it is bound by is the memory.  A thread
// takes batches of 16-byte vectors.  A warp keeps one running maximum m, so
// that a new one is rare after the first batches, and sums, over the elements
// below m,
//     s += 2^d,   w += 2^d d,   d = (x - m) * scale * log2 e,
// and counts those equal to m.  So the largest term, 1, never enters a sum: log(1 +
// s) and the entropy keep their bits where s is small.
//
// Top alternatives.  Each thread also leaves the largest element of every bucket
// of its batches (up to 32 buckets) in shared memory.  If each of the eight warps
// has ceil(k / 8) threads whose largest element is at least t, the k-th largest
// element of the block's part is at least t; only buckets that may hold an element
// of at least t are read again, some 2 k of 5000 in ordinary rows, eight at a time.
//
// 1024 rows of 151552: fp32 94 us (0.97 of the copy rate), top 1 or 20 107 (0.86); BF16
// 62 (0.74: six instructions an element), top 20 83.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "cluster.cuh"
#include "host_shared.cuh"
#include "pairs.cuh"

namespace wc {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
// Vectors of a batch and blocks an SM: 8192 rows of 8192 fp32 logits, top 20, at 8 and
// 4 126, at 6 and 4 140, at 5 and 5 147 us; 1024 of 151552 BF16 at 4 and 4 83, at 6 and
// 4 92, at 4 and 5 88.
template <bool BF16>
struct Batch {
  static constexpr int kVecs = BF16 ? 4 : 8, kBlocks = 4;
};
constexpr int kBuckets = 32;
constexpr int kMaxTop = 64;
constexpr int kMaxTeam = 8;    // blocks that share a row
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct LogprobArgs {
  const void* logits;
  const int64_t* ids;
  float* logprob;
  float* entropy;
  float* lse;
  float* top_logprobs;
  int32_t* top_ids;
  int64_t T, V, row;
  int top_k;
  float scale;
};

template <bool BF16>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
  if (BF16) return __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i]) << 16);
  return static_cast<const float*>(p)[i];
}

// A logit and its index as a number that orders as they do: NaN lowest, -0 and 0
// alike, the lower index first.  Never 0.
__device__ __forceinline__ uint64_t logit_key(float x, uint32_t i) {
  const uint32_t u = __float_as_uint(x + 0.f);
  uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) k = 0;
  return uint64_t(k) << 32 | uint32_t(~i);
}

__device__ __forceinline__ float key_logit(uint64_t key) {
  const uint32_t k = uint32_t(key >> 32);
  return k == 0 ? NAN : __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
__device__ __forceinline__ uint64_t warp_max64(uint64_t x) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, uint32_t(x >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, uint32_t(x >> 32) == hi ? uint32_t(x) : 0u);
  return uint64_t(hi) << 32 | lo;
}

// Sums relative to m: of the elements below it, and the number of those equal to it.
struct Stats {
  float m, s, w, n;
  // Go over to a larger maximum.
  __device__ __forceinline__ void raise(float to, float c) {
    if (m > -INFINITY) {
      const float by = (m - to) * c, f = exp2f(by);
      s += n;
      w = f == 0.f ? 0.f * s : f * (w + by * s);  // by may be -inf, s a NaN
      s *= f;
    }
    n = 0.f;
    m = to;
  }
};

// The sums of a list of N <= 32, by the whole warp.
__device__ __forceinline__ Stats join(const Stats* list, uint32_t n, int lane, float c) {
  Stats x{-INFINITY, 0.f, 0.f, 0.f};
  if (uint32_t(lane) < n) x = list[lane];
  const float m = warp_max(x.m);
  if (m > x.m) x.raise(m, c);
  return {m, warp_sum(x.s), warp_sum(x.w), warp_sum(x.n)};
}

// The address that a place of this block's shared memory has in the cluster's first.
__device__ __forceinline__ uint32_t in_first(const void* p) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
  return a;
}
__device__ __forceinline__ void st_cluster(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

constexpr int kList = 128;   // candidates of a warp
constexpr int kLook = 64;    // buckets that it may read again,
constexpr uint32_t kAtOnce = 8;  // so many at a time

// The loads in flight need L1, which shares its memory with this.
struct Shared {
  union {
    float top[kBuckets][kThreads];   // largest element of a thread's bucket
    uint64_t all[kWarps * kList];    // then the candidates one behind the other, in any order
  };
  uint64_t list[kWarps * kList];   // each warp's candidates; then the cluster's blocks'
  uint64_t found[kMaxTop];
  uint16_t buckets[kWarps][kLook]; // bucket and lane of those a warp reads again
  uint64_t bound[kWarps];
  uint32_t total;                  // candidates
};

// Where the elements of a block's part are.
struct Part {
  const uint8_t* z;
  uint32_t head, v0, v1, group, buckets;
};
// Index of element e of a thread's bucket, or none.
constexpr uint32_t kNoIndex = 0xFFFFFFFFu;
template <bool BF16>
__device__ __forceinline__ uint32_t part_index(const Part& p, uint32_t bucket, uint32_t owner, uint32_t e) {
  constexpr uint32_t E = BF16 ? 8 : 4, kVecs = Batch<BF16>::kVecs;
  const uint32_t v = p.v0 + (bucket * p.group * kVecs + e / E) * kThreads + owner;
  return e >= p.group * kVecs * E || v >= p.v1 ? kNoIndex : p.head + v * E + e % E;
}
// No element of the thread's bucket is larger than this.
template <bool BF16>
__device__ __forceinline__ uint64_t bucket_key(const Part& p, const Shared& sh, uint32_t bucket) {
  constexpr uint32_t kVecs = Batch<BF16>::kVecs;
  return logit_key(sh.top[bucket][threadIdx.x],
                   p.head + (p.v0 + bucket * p.group * (kThreads * kVecs) + threadIdx.x) * (BF16 ? 8 : 4));
}

// A warp's `keep` largest, where more elements than the lists take come into
// question (rows with few different values, or almost all masked): one bucket after
// the other, the list cut back whenever it is full.  Returns how many there are.
template <bool BF16>
__device__ __noinline__ uint32_t search_all(const Part& p, Shared& sh, uint64_t least, int keep) {
  constexpr uint32_t kVecs = Batch<BF16>::kVecs;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t* const list = sh.list + warp * kList;
  int count = 0;
#pragma unroll 1
  for (uint32_t b = 0; b < p.buckets; ++b) {
#pragma unroll 1
    for (uint32_t who = __ballot_sync(0xffffffffu, bucket_key<BF16>(p, sh, b) > least); who; who &= who - 1) {
#pragma unroll 1
      for (uint32_t e = lane; e - lane < p.group * kVecs * (BF16 ? 8 : 4); e += 32) {
        const uint32_t i = part_index<BF16>(p, b, uint32_t(warp * 32 + __ffs(int(who)) - 1), e);
        const uint64_t k = i == kNoIndex ? 0 : logit_key(logit<BF16>(p.z, i), i);
        const uint32_t some = __ballot_sync(0xffffffffu, k > least);
        if (k > least) list[count + __popc(some & ((1u << lane) - 1u))] = k;
        count += __popc(some);
        __syncwarp();
        if (count <= kList - 32) continue;
        uint64_t mine[kList / 32];
        int rank[kList / 32] = {};
#pragma unroll
        for (int i = 0; i < kList / 32; ++i) mine[i] = lane + 32 * i < count ? list[lane + 32 * i] : 0;
#pragma unroll 1
        for (int j = 0; j < count; ++j) {
          const uint64_t x = list[j];
#pragma unroll
          for (int i = 0; i < kList / 32; ++i) rank[i] += x > mine[i];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kList / 32; ++i)
          if (mine[i] && rank[i] < keep) list[rank[i]] = mine[i];
        __syncwarp();
        count = min(count, keep);
        if (list[keep - 1] > least) least = list[keep - 1];
        __syncwarp();
      }
    }
  }
  return uint32_t(count);
}

// The `keep` largest of list[0 .. n) but zeros, descending, to found.
__device__ __forceinline__ void rank_list(Shared& sh, const uint64_t* list, int n, int keep) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t k = list[i];
    if (!k) continue;
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += list[j] > k;
    if (rank < keep) sh.found[rank] = k;
  }
}

template <bool BF16, bool TOP>
__global__ void __launch_bounds__(kThreads, Batch<BF16>::kBlocks) logprobs_kernel(const __grid_constant__ LogprobArgs a, uint32_t team) {
  constexpr int E = BF16 ? 8 : 4;  // elements of a vector
  constexpr int kVecs = Batch<BF16>::kVecs;
  using Lists = std::conditional_t<TOP, Shared, char>;
  __shared__ Stats s_stats[kWarps > kMaxTeam ? kWarps : kMaxTeam];
  __shared__ Lists sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = team > 1 ? cluster_rank() : 0;
  const int64_t t = blockIdx.x / team;
  const uint8_t* z = static_cast<const uint8_t*>(a.logits) + t * a.row * (BF16 ? 2 : 4);
  const float c = a.scale * kLog2e;
  // elements before the first whole vector, whole vectors (this block's: v0 .. v1), elements behind
  const uint32_t V = uint32_t(a.V);
  const uint32_t head = min(V, uint32_t(-reinterpret_cast<uintptr_t>(z) & 15u) / (BF16 ? 2u : 4u));
  const uint32_t vecs = (V - head) / E, tail = head + vecs * E;
  const uint32_t v0 = uint32_t(uint64_t(vecs) * rank / team), v1 = uint32_t(uint64_t(vecs) * (rank + 1) / team);
  const uint32_t rounds = (v1 - v0 + kThreads * kVecs - 1) / (kThreads * kVecs);
  const uint32_t group = (rounds + kBuckets - 1) / kBuckets;  // batches of a bucket
  const uint8_t* zv = z + head * (BF16 ? 2 : 4);

  // the given token's logit, long before it is wanted
  int64_t id = -1;
  float given = NAN;
  if (a.ids && threadIdx.x == 0 && rank == 0) {
    id = a.ids[t];
    if (id >= 0 && id < a.V) given = logit<BF16>(z, id);
  }
  Stats st{-INFINITY, 0.f, 0.f, 0.f};
  float from = 0.f;  // m, but 0 while there is no element above -inf
  // Add a batch of N elements; `most`: their largest.
  auto add = [&](auto get, auto count, float most) {
    constexpr int N = decltype(count)::value;
    // -inf gives 0 without a NaN, a NaN stays one
    auto below = [&](float x) { return max_nan((x - from) * c, -200.f); };
    const float all = warp_max(most);
    if (all > st.m) {
      st.raise(all, c);
      from = all;
    }
    if (N % 2 == 0 && (all < st.m || st.m == -INFINITY)) {
      // two elements an instruction, in two sums
      const uint64_t minus = pair(-from, -from), c2 = pair(c, c);
      uint64_t s2 = pair(st.s, 0.f), w2 = pair(st.w, 0.f);
#pragma unroll
      for (int i = 0; i + 1 < N; i += 2) {
        const uint64_t x = mul2(add2(pair(get(i), get(i + 1)), minus), c2);
        const uint64_t d = pair(max_nan(first(x), -200.f), max_nan(second(x), -200.f));
        const uint64_t e = pair(exp2_approx(first(d)), exp2_approx(second(d)));
        s2 = add2(s2, e);
        w2 = fma2(e, d, w2);
      }
      st.s = first(s2) + second(s2);
      st.w = first(w2) + second(w2);
    } else if (all < st.m || st.m == -INFINITY) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = below(get(i)), e = exp2_approx(d);
        st.s += e;
        st.w = __fmaf_rn(e, d, st.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float x = get(i), d = below(x), e = x == st.m ? 0.f : exp2_approx(d);
        st.s += e;
        st.w = __fmaf_rn(e, d, st.w);
        st.n += x == st.m ? 1.f : 0.f;
      }
    }
  };
  using Count = std::integral_constant<int, kVecs * E>;
  using One = std::integral_constant<int, 1>;

  // the largest of the thread's buckets, and the last index of the first that has it
  float best = -INFINITY;
  uint32_t best_at = 0;
  {
    float top = -INFINITY;
    uint32_t in = 0, bucket = 0;
    for (uint32_t round = 0; round < rounds; ++round) {
      uint32_t x[kVecs][4];
      const uint32_t v = v0 + round * (kThreads * kVecs) + threadIdx.x;
      constexpr uint32_t kNone = BF16 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        uint4 y = make_uint4(kNone, kNone, kNone, kNone);
        if (v + j * kThreads < v1) y = ld_stream_v4(zv + uint64_t(v + j * kThreads) * 16);
        x[j][0] = y.x; x[j][1] = y.y; x[j][2] = y.z; x[j][3] = y.w;
      }
      auto get = [&](int i) {
        if constexpr (BF16) {
          const uint32_t word = x[i / 8][i / 2 % 4];
          return i % 2 ? bf16_hi(word) : bf16_lo(word);
        } else {
          return __uint_as_float(x[i / 4][i % 4]);
        }
      };
      float most = -INFINITY;
#pragma unroll
      for (int i = 0; i < kVecs * E; ++i) most = fmaxf(most, get(i));
      if constexpr (TOP) {
        top = fmaxf(top, most);
        if (++in == group || round + 1 == rounds) {
          sh.top[bucket][threadIdx.x] = top;
          if (top > best) {
            best = top;
            best_at = head + (v + (kVecs - 1) * kThreads) * E + E - 1;
          }
          top = -INFINITY;
          in = 0;
          ++bucket;
        }
      }
      add(get, Count{}, most);
    }
  }
  // what is not in whole vectors: the first block's
  const uint32_t edges = rank == 0 ? head + (V - tail) : 0;
  const uint32_t edge = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
  const float edge_x = threadIdx.x < edges ? logit<BF16>(z, edge) : -INFINITY;
  if (uint32_t(warp) * 32 < edges) add([&](int) { return edge_x; }, One{}, edge_x == edge_x ? edge_x : -INFINITY);

  st.s = warp_sum(st.s);
  st.w = warp_sum(st.w);
  st.n = warp_sum(st.n);
  if (lane == 0) s_stats[warp] = st;
  if constexpr (TOP) {
    const int keep = a.top_k;
    // a bound that ceil(keep / 8) threads of every warp reach
    uint64_t mine = best > -INFINITY ? logit_key(best, best_at) : 0, reached = 0;
    for (int i = 0; i < (keep + kWarps - 1) / kWarps; ++i) {
      reached = warp_max64(mine);
      if (mine == reached) mine = 0;
    }
    if (lane == 0) sh.bound[warp] = reached;
    if (threadIdx.x == 0) sh.total = 0;
    for (int i = threadIdx.x; i < keep; i += kThreads) sh.found[i] = 0;
    __syncthreads();
    st = join(s_stats, kWarps, lane, c);
    uint64_t bound = sh.bound[0];
    for (int w = 1; w < kWarps; ++w) bound = min(bound, sh.bound[w]);
    const uint64_t least = bound ? bound - 1 : 0;
    const Part part{z, head, v0, v1, group, group ? (rounds + group - 1) / group : 0};
    uint64_t* const list = sh.list + warp * kList;
    const float floor = bound ? key_logit(bound) : -INFINITY;
    uint32_t look = 0;  // buckets of this thread that may have such an element
#pragma unroll 8
    for (uint32_t b = 0; b < part.buckets; ++b) look |= uint32_t(sh.top[b][threadIdx.x] >= floor) << b;
    uint32_t listed = __popc(look);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, listed, d);
      if (lane >= d) listed += y;
    }
    for (uint32_t at = listed - __popc(look); look && at < kLook; ++at, look &= look - 1)
      sh.buckets[warp][at] = uint16_t((__ffs(int(look)) - 1) * 32 + lane);
    listed = __shfl_sync(0xffffffffu, listed, 31);
    __syncwarp();
    uint32_t count = 0;
    // lanes with an element that may be one: to the list
    auto take = [&](bool may, float x, uint32_t i) {
      if (!__any_sync(0xffffffffu, may)) return;
      const uint64_t k = may && i != kNoIndex ? logit_key(x, i) : 0;
      const uint32_t who = __ballot_sync(0xffffffffu, k > least), at = count + __popc(who & ((1u << lane) - 1u));
      if (k > least && at < kList) list[at] = k;
      count += __popc(who);
    };
    for (uint32_t b0 = 0; b0 < min(listed, uint32_t(kLook)); b0 += kAtOnce)
      for (uint32_t e0 = 0; e0 < group * kVecs * E; e0 += 32) {
        auto index = [&](uint32_t j) {
          const uint32_t which = sh.buckets[warp][min(b0 + j, listed - 1)];
          return b0 + j < listed ? part_index<BF16>(part, which / 32, uint32_t(warp) * 32 + which % 32, e0 + lane) : kNoIndex;
        };
        float x[kAtOnce];
#pragma unroll
        for (uint32_t j = 0; j < kAtOnce; ++j) {
          const uint32_t i = index(j);
          x[j] = i == kNoIndex ? -INFINITY : logit<BF16>(z, i);
        }
#pragma unroll
        for (uint32_t j = 0; j < kAtOnce; ++j) take(!(x[j] < floor), x[j], index(j));
      }
    if (uint32_t(warp) * 32 < edges) take(threadIdx.x < edges, edge_x, edge);
    __syncwarp();
    if (listed > kLook || count > kList) {
      count = search_all<BF16>(part, sh, least, keep);
      // the first warp's edges: the list has room for them
      if (uint32_t(warp) * 32 < edges) {
        if (threadIdx.x < edges) list[count + threadIdx.x] = logit_key(edge_x, edge);
        count += edges;
      }
    }
    __syncwarp();
    uint32_t place = 0;
    if (lane == 0) place = atomicAdd(&sh.total, count);
    place = __shfl_sync(0xffffffffu, place, 0);
    __syncthreads();  // nobody looks at the buckets any more
    for (uint32_t i = lane; i < count; i += 32) sh.all[place + i] = list[i];
    __syncthreads();
    rank_list(sh, sh.all, int(sh.total), keep);
    __syncthreads();
  } else {
    __syncthreads();
    st = join(s_stats, kWarps, lane, c);
  }

  if (team > 1) {
    // everything to the cluster's first block, whose lists are free once all are here
    cluster_sync();
    if (threadIdx.x == 0) {
      const uint32_t to = in_first(&s_stats[rank]);
      st_cluster(to, __float_as_uint(st.m));
      st_cluster(to + 4, __float_as_uint(st.s));
      st_cluster(to + 8, __float_as_uint(st.w));
      st_cluster(to + 12, __float_as_uint(st.n));
    }
    if constexpr (TOP) {
      const uint32_t* mine = reinterpret_cast<const uint32_t*>(sh.found);
      for (int i = threadIdx.x; i < 2 * a.top_k; i += kThreads)
        st_cluster(in_first(&sh.list[rank * a.top_k]) + 4 * i, mine[i]);
    }
    cluster_sync();
    if (rank) return;
    st = join(s_stats, team, lane, c);
    if constexpr (TOP) {
      for (int i = threadIdx.x; i < a.top_k; i += kThreads) sh.found[i] = 0;
      __syncthreads();
      rank_list(sh, sh.list, int(team) * a.top_k, a.top_k);
      __syncthreads();
    }
  }

  const float rest = st.s + (st.n - 1.f);
  const float log_sum = isfinite(st.m) ? log1pf(rest) : NAN;  // lse - scale * m
  if (threadIdx.x == 0) {
    if (a.lse) a.lse[t] = st.m * a.scale + log_sum;
    if (a.entropy) a.entropy[t] = log_sum - st.w * kLn2 / (1.f + rest);
    if (a.ids) a.logprob[t] = id < 0 ? 0.f : (given - st.m) * a.scale - log_sum;
  }
  if constexpr (TOP) {
    for (int i = threadIdx.x; i < a.top_k; i += kThreads) {
      a.top_ids[t * a.top_k + i] = int32_t(~uint32_t(sh.found[i]));
      a.top_logprobs[t * a.top_k + i] = (key_logit(sh.found[i]) - st.m) * a.scale - log_sum;
    }
  }
}

template <bool BF16, bool TOP>
cudaError_t launch(const LogprobArgs& a, uint32_t team, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(uint32_t(a.T) * team);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = team;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = team > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<BF16, TOP>, a, team);
}

}  // namespace
}  // namespace wc

using namespace wc;

extern "C" int wcomp_logprobs(const wcomp_logprobs_args* args, void* stream) {
  if (!args) return WCOMP_EINVAL;
  const wcomp_logprobs_args& a = *args;
  if (a.T < 0 || a.V < 1 || a.row < a.V || (a.dtype != WCOMP_FP32 && a.dtype != WCOMP_BF16) || a.top_k < 0 ||
      a.top_k > a.V || !(a.scale > 0.f) || !std::isfinite(a.scale * kLog2e) || (a.T && !a.d_logits) ||
      (a.T && a.top_k && (!a.d_top_logprobs || !a.d_top_ids)) || (a.T && a.d_ids && !a.d_logprob))
    return WCOMP_EINVAL;
  if (reinterpret_cast<uintptr_t>(a.d_logits) % (a.dtype == WCOMP_BF16 ? 2 : 4) || !natural(a.d_ids) || !natural(a.d_logprob) ||
      !natural(a.d_entropy) || !natural(a.d_lse) || !natural(a.d_top_logprobs) || !natural(a.d_top_ids))
    return WCOMP_EINVAL;
  if (a.top_k > kMaxTop || a.V >= (int64_t(1) << 31) || a.T >= (int64_t(1) << 28)) return WCOMP_EUNSUPPORTED;
  if (a.T == 0) return WCOMP_OK;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return map_cuda(cudaGetLastError());
  const LogprobArgs p{a.d_logits, a.d_ids,  a.d_logprob, a.d_entropy, a.d_lse, a.d_top_logprobs, a.d_top_ids,
                      a.T,        a.V,      a.row,       a.top_k,     a.scale};
  // Blocks share a row while that leaves them a batch each and two blocks an SM take all
  // rows.  151552 fp32 logits, us by 1, 2, 4 and 8 blocks: 16 rows 14.6, 12.4, 8.3, 8.3;
  // 76 rows 16.4, 12.3, 12.4, 14.3; 152 rows 22.5, 16.5, 20.1, 22.4; 400 rows 39.6, 51.5.
  uint32_t team = 1;
  const int64_t batch = int64_t(kThreads) * (a.dtype == WCOMP_BF16 ? Batch<true>::kVecs * 8 : Batch<false>::kVecs * 4);
  while (team < kMaxTeam && a.T * team * 2 <= sm_count(dev) * 2 && a.V >= batch * team * 2) team *= 2;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.dtype == WCOMP_BF16
                            ? (a.top_k ? launch<true, true>(p, team, s) : launch<true, false>(p, team, s))
                            : (a.top_k ? launch<false, true>(p, team, s) : launch<false, false>(p, team, s));
  count_launches(1);
  return map_cuda(e);
}
