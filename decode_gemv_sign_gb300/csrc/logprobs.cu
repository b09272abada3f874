// Log probabilities, entropy and top alternatives from logits.
//
// A row is read once, by a block of 256 threads or, where there are few rows, by a
// cluster of blocks that share it; what it is bound by is the memory.  A thread
// takes batches of four 16-byte vectors.  A warp keeps one running maximum m, so
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
// of at least t are read again, some 2 k of 8192 in ordinary rows.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "wcomp_impl.cuh"

namespace wc {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVecs = 4;       // vectors of a batch
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

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int d = 16; d; d /= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
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
  __device__ __forceinline__ void add(const Stats& o, float c) {
    Stats x = o;
    if (x.m > m) raise(x.m, c);
    if (m > x.m) x.raise(m, c);
    s += x.s;
    w += x.w;
    n += x.n;
  }
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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

// A warp's largest keys, two a lane, in no order.
struct Best {
  uint64_t key[2] = {0, 0}, least = 0;  // least: below it nothing enters
  __device__ __forceinline__ void offer(uint64_t k, int keep, int lane) {
    for (uint32_t who; (who = __ballot_sync(0xffffffffu, k > least)) != 0;) {
      const int from = __ffs(int(who)) - 1;
      const uint64_t x = __shfl_sync(0xffffffffu, k, from);
      if (lane == from) k = 0;
      // takes the place of the least of `keep` places
      const bool second = lane + 32 < keep;
      uint64_t mine = lane < keep ? key[0] : ~uint64_t(0);
      if (second && key[1] < mine) mine = key[1];
      const uint64_t low = ~warp_max64(~mine);
      const int at = __ffs(int(__ballot_sync(0xffffffffu, mine == low))) - 1;
      if (lane == at) {
        if (key[0] == low) key[0] = x;
        else key[1] = x;
      }
      mine = lane < keep ? key[0] : ~uint64_t(0);
      if (second && key[1] < mine) mine = key[1];
      const uint64_t now = ~warp_max64(~mine);
      if (now > least) least = now;
    }
  }
};

struct Shared {
  float top[kBuckets][kThreads];  // largest element of a thread's bucket
  Stats stats[kWarps > kMaxTeam ? kWarps : kMaxTeam];
  uint64_t list[kWarps * kMaxTop];
  uint64_t found[kMaxTop];
  uint64_t bound[kWarps];
  uint32_t count;
};

// The `keep` largest of list[0 .. n), descending, to found; what is missing is 0.
__device__ __forceinline__ void rank_list(Shared& sh, int n, int keep) {
  for (int i = threadIdx.x; i < keep; i += kThreads) sh.found[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t k = sh.list[i];
    if (!k) continue;
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += sh.list[j] > k;
    if (rank < keep) sh.found[rank] = k;
  }
  __syncthreads();
}

template <bool BF16, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const __grid_constant__ LogprobArgs a, uint32_t team) {
  constexpr int E = BF16 ? 8 : 4;  // elements of a vector
  __shared__ Shared sh;
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
    if (all < st.m || st.m == -INFINITY) {
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
  if (lane == 0) sh.stats[warp] = st;
  __syncthreads();
  st = sh.stats[0];
  for (int w = 1; w < kWarps; ++w) st.add(sh.stats[w], c);

  if constexpr (TOP) {
    const int keep = a.top_k;
    // a bound that ceil(keep / 8) threads of every warp reach
    uint64_t mine = best > -INFINITY ? logit_key(best, best_at) : 0, reached = 0;
    for (int i = 0; i < (keep + kWarps - 1) / kWarps; ++i) {
      reached = warp_max64(mine);
      if (mine == reached) mine = 0;
    }
    if (lane == 0) sh.bound[warp] = reached;
    __syncthreads();
    uint64_t bound = sh.bound[0];
    for (int w = 1; w < kWarps; ++w) bound = min(bound, sh.bound[w]);
    Best mostly;
    mostly.least = bound ? bound - 1 : 0;
    const uint32_t buckets = group ? (rounds + group - 1) / group : 0;
    for (uint32_t b = 0; b < buckets; ++b) {
      // no element of the bucket is larger than this
      const uint32_t low = head + (v0 + b * group * (kThreads * kVecs) + threadIdx.x) * E;
      uint32_t who = __ballot_sync(0xffffffffu, logit_key(sh.top[b][threadIdx.x], low) > mostly.least);
      for (; who; who &= who - 1) {
        const uint32_t owner = uint32_t(warp) * 32 + uint32_t(__ffs(int(who))) - 1;
        const uint32_t n = group * kVecs * E;
        for (uint32_t e0 = 0; e0 < n; e0 += 32) {
          const uint32_t e = e0 + lane, v = v0 + (b * group * kVecs + e / E) * kThreads + owner;
          uint64_t k = 0;
          if (e < n && v < v1) {
            const uint32_t i = head + v * E + e % E;
            k = logit_key(logit<BF16>(z, i), i);
          }
          mostly.offer(k, keep, lane);
        }
      }
    }
    if (uint32_t(warp) * 32 < edges)
      mostly.offer(threadIdx.x < edges ? logit_key(edge_x, edge) : 0, keep, lane);
    // the warps' keys together, those that are there
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (mostly.key[i]) sh.list[atomicAdd(&sh.count, 1u)] = mostly.key[i];
    __syncthreads();
    rank_list(sh, int(sh.count), keep);
  }

  if (team > 1) {
    // everything to the cluster's first block, whose lists are free once all are here
    cluster_sync();
    if (threadIdx.x < 4) {
      const float v[4] = {st.m, st.s, st.w, st.n};
      st_cluster(in_first(&sh.stats[rank]) + 4 * threadIdx.x, __float_as_uint(v[threadIdx.x]));
    }
    if constexpr (TOP) {
      const uint32_t* mine = reinterpret_cast<const uint32_t*>(sh.found);
      for (int i = threadIdx.x; i < 2 * a.top_k; i += kThreads)
        st_cluster(in_first(&sh.list[rank * a.top_k]) + 4 * i, mine[i]);
    }
    cluster_sync();
    if (rank) return;
    st = sh.stats[0];
    for (uint32_t w = 1; w < team; ++w) st.add(sh.stats[w], c);
    if constexpr (TOP) rank_list(sh, int(team) * a.top_k, a.top_k);
  }

  const float rest = st.s + (st.n - 1.f);
  const float log_sum = isfinite(st.m) ? log1pf(rest) : NAN;  // lse - scale * m
  if (threadIdx.x == 0) {
    if (a.lse) a.lse[t] = st.m * a.scale + log_sum;
    if (a.entropy) a.entropy[t] = log_sum - st.w * kLn2 / (1.f + rest);
    if (a.ids) {
      const int64_t id = a.ids[t];
      a.logprob[t] = id < 0 ? 0.f : id >= a.V ? NAN : (logit<BF16>(z, id) - st.m) * a.scale - log_sum;
    }
  }
  if constexpr (TOP) {
    for (int i = threadIdx.x; i < a.top_k; i += kThreads) {
      const uint32_t id = ~uint32_t(sh.found[i]);
      a.top_ids[t * a.top_k + i] = int32_t(id);
      a.top_logprobs[t * a.top_k + i] = (logit<BF16>(z, id) - st.m) * a.scale - log_sum;
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
      a.top_k > a.V || !(a.scale > 0.f) || !std::isfinite(a.scale) || (a.T && !a.d_logits) ||
      (a.T && a.top_k && (!a.d_top_logprobs || !a.d_top_ids)) || (a.T && a.d_ids && !a.d_logprob))
    return WCOMP_EINVAL;
  if (a.top_k > kMaxTop || a.V >= (int64_t(1) << 31) || a.T >= (int64_t(1) << 28)) return WCOMP_EUNSUPPORTED;
  if (a.T == 0) return WCOMP_OK;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return map_cuda(cudaGetLastError());
  const LogprobArgs p{a.d_logits, a.d_ids,  a.d_logprob, a.d_entropy, a.d_lse, a.d_top_logprobs, a.d_top_ids,
                      a.T,        a.V,      a.row,       a.top_k,     a.scale};
  // blocks share a row while that leaves them a batch each and fits the GPU at once
  uint32_t team = 1;
  const int64_t batch = int64_t(kThreads) * kVecs * (a.dtype == WCOMP_BF16 ? 8 : 4);
  while (team < kMaxTeam && a.T * team * 2 <= sm_count(dev) * 2 && a.V >= batch * team * 2) team *= 2;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.dtype == WCOMP_BF16
                            ? (a.top_k ? launch<true, true>(p, team, s) : launch<true, false>(p, team, s))
                            : (a.top_k ? launch<false, true>(p, team, s) : launch<false, false>(p, team, s));
  count_launches(1);
  return map_cuda(e);
}
