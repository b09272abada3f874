// Attention over the 4-bit key/value cache.
#include <algorithm>
#include <cmath>

#include "kv4.cuh"

namespace wc {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct AttendArgs {
  KvSeqs s;
  const uint8_t* cache;
  const uint16_t* q;
  int64_t q_row, q_head;
  uint16_t* out;
  float* lse;
  float* mass;
  int64_t T;
  int q_heads, window;
  float scale;
};

// Code and scale of column c of token t in a block, as a value.
template <int D>
__device__ __forceinline__ float kv_value(const uint8_t* block, bool value, uint32_t t, uint32_t c) {
  using L = Kv<D>;
  const uint32_t g = c / 32, in = c % 32;
  const uint32_t word = value ? in / 4 * (L::G / 2) + g / 2 : in / 8 * L::G + g;
  const uint32_t nibble = value ? in % 4 + 4 * (g % 2) : in % 8;
  const uint32_t w =
      *reinterpret_cast<const uint32_t*>(block + (value ? L::kCodes : 0) + L::at(t, 4 * word));
  const uint32_t s = *reinterpret_cast<const uint16_t*>(block + (value ? L::kValueScales : L::kKeyScales) +
                                                        L::scale(t, g));
  return float(int((w >> (4 * nibble)) & 15) - 8) * __uint_as_float(s << 16);
}

// One warp takes a row and query head through its tokens.
template <int D>
__global__ void __launch_bounds__(kThreads) kv4_attend_kernel(AttendArgs a) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x % 32;
  const int64_t units = a.T * a.q_heads;
  const int share = a.q_heads / int(a.s.heads);
  for (int64_t unit = int64_t(blockIdx.x) * kWarps + threadIdx.x / 32; unit < units;
       unit += int64_t(gridDim.x) * kWarps) {
    const int64_t i = unit / a.q_heads;
    const int hq = int(unit % a.q_heads), h = hq / share;
    const int b = kv_sequence(a.s, i);
    if (b < 0) continue;
    const int64_t pos = kv_position(a.s, b, i, kv_length(a.s, b));
    float q[kPer], o[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      q[j] = __uint_as_float(uint32_t(a.q[i * a.q_row + hq * a.q_head + lane + 32 * j]) << 16) * a.scale;
      o[j] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const int64_t first = a.window ? max(int64_t(0), pos - a.window + 1) : 0;
    for (int64_t p = first; p <= pos; ++p) {
      const int page = kv_page(a.s, b, int(p / kPage));
      if (page < 0) continue;
      const uint8_t* block = a.cache + (uint64_t(page) * a.s.heads + h) * Kv<D>::kBlock;
      float z = 0.f;
#pragma unroll
      for (int j = 0; j < kPer; ++j) z += q[j] * kv_value<D>(block, false, p % kPage, lane + 32 * j);
#pragma unroll
      for (int d = 16; d; d /= 2) z += __shfl_xor_sync(0xffffffffu, z, d);
      const float next = fmaxf(m, z);
      const float down = m == -INFINITY ? 0.f : expf(m - next), e = expf(z - next);
      l = l * down + e;
      m = next;
#pragma unroll
      for (int j = 0; j < kPer; ++j) o[j] = o[j] * down + e * kv_value<D>(block, true, p % kPage, lane + 32 * j);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      uint16_t bits;
      asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(bits) : "f"(l == 0.f ? 0.f : o[j] / l));
      a.out[(i * a.q_heads + hq) * D + lane + 32 * j] = bits;
    }
    if (lane == 0) a.lse[i * a.q_heads + hq] = m + logf(l);
  }
}

// One warp adds to a token's weight what the rows of its sequence give it.
template <int D>
__global__ void __launch_bounds__(kThreads) kv4_mass_kernel(AttendArgs a) {
  const int lane = threadIdx.x % 32;
  const int share = a.q_heads / int(a.s.heads);
  const int64_t tokens = int64_t(a.s.width) * kPage;
  const int64_t units = int64_t(a.s.B) * a.s.heads * tokens;
  for (int64_t unit = int64_t(blockIdx.x) * kWarps + threadIdx.x / 32; unit < units;
       unit += int64_t(gridDim.x) * kWarps) {
    const int64_t p = unit % tokens;
    const int h = int(unit / tokens % a.s.heads), b = int(unit / tokens / a.s.heads);
    const int n = kv_length(a.s, b);
    if (p >= n) continue;
    const int page = kv_page(a.s, b, int(p / kPage));
    if (page < 0) continue;
    const uint8_t* block = a.cache + (uint64_t(page) * a.s.heads + h) * Kv<D>::kBlock;
    const int64_t i0 = a.s.starts ? max(0, a.s.starts[b]) : b;
    const int64_t i1 = a.s.starts ? min(a.T, int64_t(a.s.starts[b + 1])) : b + 1;
    float sum = 0.f;
    for (int64_t i = i0; i < i1; ++i) {
      const int64_t pos = kv_position(a.s, b, i, n);
      if (p > pos || (a.window && p <= pos - a.window)) continue;
      for (int hq = h * share; hq < (h + 1) * share; ++hq) {
        float z = 0.f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          z += __uint_as_float(uint32_t(a.q[i * a.q_row + hq * a.q_head + lane + 32 * j]) << 16) * a.scale *
               kv_value<D>(block, false, p % kPage, lane + 32 * j);
#pragma unroll
        for (int d = 16; d; d /= 2) z += __shfl_xor_sync(0xffffffffu, z, d);
        sum += expf(z - a.lse[i * a.q_heads + hq]);
      }
    }
    if (lane == 0) a.mass[unit] += sum;
  }
}

}  // namespace
}  // namespace wc

using namespace wc;

extern "C" int wcomp_kv4_attend(const wcomp_kv4* c, const wcomp_kv4_attend_args* args, void* stream) {
  if (!c || !args) return WCOMP_EINVAL;
  const wcomp_kv4_attend_args& a = *args;
  int st = kv_check(c, a.s, a.T);
  if (st != WCOMP_OK) return st;
  if (a.q_heads < 1 || a.q_heads % c->heads || a.window < 0 || !std::isfinite(a.scale) || a.q_row < 0 || a.q_head < 0 ||
      (a.T && (!a.d_q || !a.d_out || a.d_out == a.d_q)))
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
  p.out = a.d_out;
  p.lse = a.d_lse;
  p.mass = a.d_mass;
  p.T = a.T;
  p.q_heads = a.q_heads;
  p.window = a.window;
  p.scale = a.scale;
  void* ws = nullptr;
  const uint64_t b_lse = uint64_t(a.T) * a.q_heads * sizeof(float);
  cudaError_t e = pool_alloc(&ws, b_lse, s);
  if (e != cudaSuccess) return map_cuda(e);
  if (!p.lse) p.lse = static_cast<float*>(ws);
  const uint32_t grid = uint32_t(std::min<int64_t>(int64_t(cdiv(a.T * a.q_heads, kWarps)), sm_count(c->device) * 64));
#define CALL(D)                                                                                              \
  do {                                                                                                       \
    kv4_attend_kernel<D><<<grid, kThreads, 0, s>>>(p);                                                       \
    if (p.mass) kv4_mass_kernel<D><<<uint32_t(sm_count(c->device)) * 8, kThreads, 0, s>>>(p);                \
  } while (0)
  if (c->dim == 64) CALL(64);
  else if (c->dim == 128) CALL(128);
  else CALL(256);
#undef CALL
  e = cudaGetLastError();
  count_launches(p.mass ? 2 : 1);
  cudaFreeAsync(ws, s);
  return map_cuda(e);
}
