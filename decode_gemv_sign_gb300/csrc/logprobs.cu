// Log probabilities, entropy and top alternatives from logits.
#include <algorithm>
#include <cmath>

#include "wcomp_impl.cuh"

namespace wc {
namespace {

constexpr int kThreads = 512;

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
// alike, the lower index first.
__device__ __forceinline__ uint64_t logit_key(float x, uint32_t i) {
  const uint32_t u = __float_as_uint(x + 0.f);
  uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) k = 0;
  return uint64_t(k) << 32 | uint32_t(~i);
}

template <class T, class F>
__device__ T block_reduce(T v, F f, T* s) {
#pragma unroll
  for (int d = 16; d; d /= 2) v = f(v, __shfl_xor_sync(0xffffffffu, v, d));
  __syncthreads();
  if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = v;
  __syncthreads();
  v = s[0];
  for (int w = 1; w < kThreads / 32; ++w) v = f(v, s[w]);
  return v;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(LogprobArgs a) {
  __shared__ uint64_t s_key[kThreads / 32];
  __shared__ float s_sum[kThreads / 32];
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const void* z = static_cast<const uint8_t*>(a.logits) + t * a.row * (BF16 ? 2 : 4);
    auto larger = [](uint64_t x, uint64_t y) { return x > y ? x : y; };
    auto plus = [](float x, float y) { return x + y; };
    uint64_t best = 0;
    for (int64_t i = threadIdx.x; i < a.V; i += kThreads) best = larger(best, logit_key(logit<BF16>(z, i), uint32_t(i)));
    best = block_reduce(best, larger, s_key);
    const uint32_t at = ~uint32_t(best);
    const float m = logit<BF16>(z, at);
    // the largest term is left out until the end
    float rest = 0.f, weighted = 0.f;
    for (int64_t i = threadIdx.x; i < a.V; i += kThreads) {
      if (i == at) continue;
      const float d = (logit<BF16>(z, i) - m) * a.scale, e = expf(d);
      rest += e;
      if (e != 0.f) weighted += e * d;
    }
    rest = block_reduce(rest, plus, s_sum);
    weighted = block_reduce(weighted, plus, s_sum);
    const float log_sum = isfinite(m) ? log1pf(rest) : NAN;  // lse - scale * m
    if (threadIdx.x == 0) {
      if (a.lse) a.lse[t] = m * a.scale + log_sum;
      if (a.entropy) a.entropy[t] = log_sum - weighted / (1.f + rest);
      if (a.ids) {
        const int64_t id = a.ids[t];
        a.logprob[t] = id < 0 ? 0.f : id >= a.V ? NAN : (logit<BF16>(z, id) - m) * a.scale - log_sum;
      }
    }
    for (int k = 0; k < a.top_k; ++k) {
      if (threadIdx.x == 0) {
        a.top_ids[t * a.top_k + k] = int32_t(~uint32_t(best));
        a.top_logprobs[t * a.top_k + k] = (logit<BF16>(z, ~uint32_t(best)) - m) * a.scale - log_sum;
      }
      const uint64_t last = best;
      best = 0;
      for (int64_t i = threadIdx.x; i < a.V; i += kThreads) {
        const uint64_t key = logit_key(logit<BF16>(z, i), uint32_t(i));
        if (key < last) best = larger(best, key);
      }
      best = block_reduce(best, larger, s_key);
    }
  }
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
  if (a.top_k > 64 || a.V >= (int64_t(1) << 31)) return WCOMP_EUNSUPPORTED;
  if (a.T == 0) return WCOMP_OK;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return map_cuda(cudaGetLastError());
  const LogprobArgs p{a.d_logits, a.d_ids,  a.d_logprob, a.d_entropy, a.d_lse, a.d_top_logprobs, a.d_top_ids,
                      a.T,        a.V,      a.row,       a.top_k,     a.scale};
  const uint32_t grid = uint32_t(std::min<int64_t>(a.T, sm_count(dev) * 16));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.dtype == WCOMP_BF16) logprobs_kernel<true><<<grid, kThreads, 0, s>>>(p);
  else logprobs_kernel<false><<<grid, kThreads, 0, s>>>(p);
  count_launches(1);
  return map_cuda(cudaGetLastError());
}
