// Writing, reading and evicting from the 4-bit key/value cache.
#include <algorithm>
#include <new>

#include "kv4.cuh"

namespace wc {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ uint32_t bf16_bits(float v) {
  uint16_t h;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
  return h;
}

// A row of keys or values is handled by D / 8 neighbouring threads, thread u the
// columns 8 u .. 8 u + 7; four of them share a group.  The threads of a row are in
// one warp, which handles 256 / D rows at a time.
template <int D>
struct RowThreads {
  static constexpr int kPer = D / 8;
  static constexpr int kRows = kThreads / kPer;  // of a block
};

// Quantise 8 columns; four lanes share the group's largest magnitude.  `w` gets the
// codes, 4 bits each; returns the scale's bits.
__device__ __forceinline__ uint32_t quantise8(const uint32_t (&v)[4], uint32_t& w) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  w = 0x88888888u;
  if (m > 0x7F7Fu) return 0x7FC0u;  // an infinity or a NaN
  const uint32_t sb = bf16_bits(bf16_value(m) / 7.f);
  if (sb == 0u) return 0u;
  const float s = bf16_value(sb);
  w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = bf16_value((v[i / 2] >> (16 * (i % 2))) & 0xFFFFu);
    // a quotient of 8-bit significands is a midpoint or well off one: its fp32
    // rounding does not move it over an edge
    const int c = max(-7, min(7, __float2int_rn(x / s))) + 8;
    w |= uint32_t(c) << (4 * i);
  }
  return sb;
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

// One warp's unit: 256 / D (token, head) pairs, keys and then values of each.
template <int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(KvSeqs s, uint8_t* cache, Rows k, Rows v, int64_t T) {
  const uint32_t u = threadIdx.x % RowThreads<D>::kPer;
  const int64_t n = T * s.heads;
  const int64_t step = int64_t(gridDim.x) * RowThreads<D>::kRows;
  const int64_t rounds = (n + step - 1) / step;
  int64_t at = int64_t(blockIdx.x) * RowThreads<D>::kRows + threadIdx.x / RowThreads<D>::kPer;
  for (int64_t round = 0; round < rounds; ++round, at += step) {
    // every lane takes part in the exchanges
    const int64_t i = at / s.heads, h = at % s.heads;
    const int b = at < n ? kv_sequence(s, i) : -1;
    uint8_t* block = nullptr;
    uint32_t t = 0;
    if (b >= 0) {
      const int64_t pos = kv_position(s, b, i, kv_length(s, b));
      const int page = pos < 0 ? -1 : kv_page(s, b, int(pos / kPage));
      t = uint32_t(pos) % kPage;
      if (page >= 0) block = cache + (uint64_t(page) * s.heads + h) * Kv<D>::kBlock;
    }
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const Rows& r = part ? v : k;
      uint32_t x[4] = {0, 0, 0, 0};
      if (block) {
        const uint16_t* p = r.p + i * r.row + h * r.head + 8 * u;
        if (r.vec) {
          const uint4 y = *reinterpret_cast<const uint4*>(p);
          x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = p[2 * j] | uint32_t(p[2 * j + 1]) << 16;
        }
      }
      uint32_t w;
      const uint32_t scale = quantise8(x, w);
      if (part) w = value_word(w, u);
      if (block) {
        const uint32_t index = part ? value_index<D>(u) : key_index<D>(u);
        *reinterpret_cast<uint32_t*>(block + part * Kv<D>::kHalf + Kv<D>::at(t, 4 * index)) = w;
        if ((u & 3) == 0)
          *reinterpret_cast<uint16_t*>(block + part * Kv<D>::kHalf + Kv<D>::scale(t, u >> 2)) = uint16_t(scale);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(KvSeqs s, const uint8_t* cache, uint16_t* k, uint16_t* v,
                                                            int64_t T, int vec) {
  const uint32_t u = threadIdx.x % RowThreads<D>::kPer;
  const int64_t n = T * s.heads;
  const int64_t step = int64_t(gridDim.x) * RowThreads<D>::kRows;
  const int64_t rounds = (n + step - 1) / step;
  int64_t at = int64_t(blockIdx.x) * RowThreads<D>::kRows + threadIdx.x / RowThreads<D>::kPer;
  for (int64_t round = 0; round < rounds; ++round, at += step) {
    const int64_t i = at / s.heads, h = at % s.heads;
    const int b = at < n ? kv_sequence(s, i) : -1;
    const uint8_t* block = nullptr;
    uint32_t t = 0;
    if (b >= 0) {
      const int64_t pos = kv_position(s, b, i, kv_length(s, b));
      const int page = pos < 0 ? -1 : kv_page(s, b, int(pos / kPage));
      t = uint32_t(pos) % kPage;
      if (page >= 0) block = cache + (uint64_t(page) * s.heads + h) * Kv<D>::kBlock;
    }
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      uint32_t w = 0x88888888u, scale = 0;
      if (block) {
        const uint32_t index = part ? value_index<D>(u) : key_index<D>(u);
        w = *reinterpret_cast<const uint32_t*>(block + part * Kv<D>::kHalf + Kv<D>::at(t, 4 * index));
        scale = *reinterpret_cast<const uint16_t*>(block + part * Kv<D>::kHalf + Kv<D>::scale(t, u >> 2));
      }
      if (part) w = value_word(w, u);
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float f = bf16_value(scale);
        x[j] = bf16_bits(float(int((w >> (8 * j)) & 15) - 8) * f) |
               bf16_bits(float(int((w >> (8 * j + 4)) & 15) - 8) * f) << 16;
      }
      if (b >= 0) {
        uint16_t* p = (part ? v : k) + at * D + 8 * u;
        if (vec) {
          *reinterpret_cast<uint4*>(p) = make_uint4(x[0], x[1], x[2], x[3]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) p[j] = uint16_t(x[j / 2] >> (16 * (j % 2)));
        }
      }
    }
  }
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

constexpr int kChoose = 1024;

// A mass as a number that orders as it does: NaN lowest, -0 and 0 alike.
__device__ __forceinline__ uint32_t mass_key(float m) {
  const uint32_t u = __float_as_uint(m + 0.f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the block of a count; `total` gets the sum of all.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* s_warp, uint32_t& total) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= uint32_t(d)) x += y;
  }
  __syncthreads();  // s_warp may still be read
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint32_t y = s_warp[lane];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t z = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= uint32_t(d)) y += z;
    }
    s_warp[lane] = y;
  }
  __syncthreads();
  total = s_warp[31];
  return x - v + (warp ? s_warp[warp - 1] : 0u);
}

// The `want` largest keys of the first n0 tokens, by a radix selection of 8 bits at
// a time: the key of the last one taken, and how many of those that equal it.
__global__ void __launch_bounds__(kChoose) kv4_choose_kernel(EvictArgs a) {
  __shared__ uint32_t s_bins[256], s_warp[32], s_pick[2];
  const uint32_t tid = threadIdx.x;
  const int64_t units = int64_t(a.s.B) * a.s.heads;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int b = int(unit / a.s.heads);
    const int n = kv_length(a.s, b);
    const int m = min(n, a.keep);
    const float* mass = a.mass + unit * a.s.width * kPage;
    float* mass_out = a.mass_out + unit * a.width_out * kPage;
    int32_t* kept = a.kept + unit * a.keep;
    if (unit % a.s.heads == 0 && tid == 0) a.lengths_out[b] = m;
    const int n0 = m < n ? n - a.recent : 0;         // tokens to choose from; those behind are kept
    uint32_t want = m < n ? uint32_t(a.keep - a.recent) : 0u;
    uint32_t prefix = 0, ties = 0;
    if (want) {
      for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) s_bins[tid] = 0;
        __syncthreads();
        for (int i = int(tid); i < n0; i += kChoose) {
          const uint32_t k = mass_key(mass[i]);
          if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&s_bins[(k >> shift) & 255], 1u);
        }
        __syncthreads();
        if (tid == 0) {
          uint32_t left = want;
          int d = 255;
          while (d > 0 && s_bins[d] < left) left -= s_bins[d--];
          s_pick[0] = uint32_t(d);
          s_pick[1] = left;
        }
        __syncthreads();
        prefix = prefix << 8 | s_pick[0];
        want = s_pick[1];
      }
      ties = want;
    }
    // in order: above the last key, or equal to it while there are some to take
    uint32_t done = 0, seen = 0;
    for (int i0 = 0; i0 < n; i0 += kChoose) {
      const int i = i0 + int(tid);
      const float x = i < n ? mass[i] : 0.f;
      const uint32_t k = mass_key(x);
      const bool tie = i < n0 && ties && k == prefix;
      uint32_t all_ties = 0, all = 0;
      const uint32_t before = block_scan(tie, s_warp, all_ties);
      const bool take = i < n && (m == n || i >= n0 || (ties && k > prefix) || (tie && seen + before < ties));
      const uint32_t place = done + block_scan(take, s_warp, all);
      if (take) {
        kept[place] = i;
        mass_out[place] = x;
      }
      done += all;
      seen += all_ties;
    }
    for (int i = m + int(tid); i < a.keep; i += kChoose) kept[i] = -1;
    for (int i = m + int(tid); i < a.width_out * kPage; i += kChoose) mass_out[i] = 0.f;
    __syncthreads();
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_move_kernel(EvictArgs a) {
  using L = Kv<D>;
  __shared__ int64_t s_src[kPage];  // the block's source, or -1, and the token in it
  __shared__ uint32_t s_at[kPage];
  const int64_t tiles = (a.keep + kPage - 1) / kPage;
  const int64_t units = int64_t(a.s.B) * a.s.heads * tiles;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t bh = unit / tiles;
    const int tile = int(unit % tiles), b = int(bh / a.s.heads), h = int(bh % a.s.heads);
    __syncthreads();
    if (threadIdx.x < kPage) {
      const int i = tile * kPage + int(threadIdx.x);
      const int pos = i < a.keep ? a.kept[bh * a.keep + i] : -1;
      const int page = pos < 0 ? -1 : kv_page(a.s, b, pos / kPage);
      s_src[threadIdx.x] = page < 0 ? -1 : (int64_t(page) * a.s.heads + h) * L::kBlock;
      s_at[threadIdx.x] = uint32_t(pos) % kPage;
    }
    __syncthreads();
    if (a.kept[bh * a.keep + tile * kPage] < 0) continue;  // a shorter sequence: nothing here, no page needed
    const int out = a.table_out[int64_t(b) * a.width_out + tile];
    if (uint32_t(out) >= a.s.pages) {
      if (threadIdx.x == 0) kv_bad(a.s.err);
      continue;
    }
    uint8_t* dst = a.cache + (uint64_t(out) * a.s.heads + h) * L::kBlock;
    constexpr int kPieces = 2 * L::kRow / 16;  // 16-byte pieces of a token's keys and values
    for (uint32_t j = threadIdx.x; j < kPage * kPieces; j += kThreads) {
      const uint32_t t = j / kPieces, piece = j % kPieces;
      if (s_src[t] < 0) continue;
      const uint32_t part = piece / (kPieces / 2) * L::kHalf, byte = piece % (kPieces / 2) * 16;
      *reinterpret_cast<uint4*>(dst + part + L::at(t, byte)) =
          *reinterpret_cast<const uint4*>(a.cache + s_src[t] + part + L::at(s_at[t], byte));
    }
    for (uint32_t j = threadIdx.x; j < kPage * 2 * L::G; j += kThreads) {
      const uint32_t t = j % kPage, g = j / kPage % L::G, part = j / kPage / L::G * L::kHalf;
      if (s_src[t] < 0) continue;
      *reinterpret_cast<uint16_t*>(dst + part + L::scale(t, g)) =
          *reinterpret_cast<const uint16_t*>(a.cache + s_src[t] + part + L::scale(s_at[t], g));
    }
  }
}

bool on_device(const wcomp_kv4* c) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == c->device;
}

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
  if (int64_t(s.width) * kPage >= (int64_t(1) << 31) || T >= (int64_t(1) << 31)) return WCOMP_EUNSUPPORTED;
  return WCOMP_OK;
}

int kv_seqs(const wcomp_kv4* c, const wcomp_kv4_seqs& s, KvSeqs* out) {
  if (!on_device(c)) return WCOMP_EINVAL;
  *out = {s.d_table, s.d_lengths, s.d_starts, s.B, s.width, uint32_t(c->pages), uint32_t(c->heads), nullptr};
  return work_error(c->device, &out->err);
}

}  // namespace wc

using namespace wc;

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
  if (!seqs || (T && (!d_k || !d_v)) || k_row < 0 || k_head < 0 || v_row < 0 || v_head < 0) return WCOMP_EINVAL;
  int st = kv_check(c, *seqs, T);
  if (st != WCOMP_OK) return st;
  KvSeqs s;
  if ((st = kv_seqs(c, *seqs, &s)) != WCOMP_OK) return st;
  if (T == 0 || s.B == 0) return WCOMP_OK;
  const Rows k{d_k, k_row, k_head, rows_vec(d_k, k_row, k_head)}, v{d_v, v_row, v_head, rows_vec(d_v, v_row, v_head)};
#define CALL(D)                                                                                             \
  kv4_append_kernel<D><<<grid_of(cdiv(T * c->heads, RowThreads<D>::kRows), c->device), kThreads, 0,         \
                         static_cast<cudaStream_t>(stream)>>>(s, c->d, k, v, T)
  WCOMP_KV_DIM(c->dim, CALL);
#undef CALL
  count_launches(1);
  return map_cuda(cudaGetLastError());
}

extern "C" int wcomp_kv4_read(const wcomp_kv4* c, const wcomp_kv4_seqs* seqs, uint16_t* d_k, uint16_t* d_v, int64_t T,
                              void* stream) {
  if (!seqs || (T && (!d_k || !d_v))) return WCOMP_EINVAL;
  int st = kv_check(c, *seqs, T);
  if (st != WCOMP_OK) return st;
  KvSeqs s;
  if ((st = kv_seqs(c, *seqs, &s)) != WCOMP_OK) return st;
  if (T == 0 || s.B == 0) return WCOMP_OK;
  const int vec = rows_vec(d_k, 0, 0) && rows_vec(d_v, 0, 0);
#define CALL(D)                                                                                           \
  kv4_read_kernel<D><<<grid_of(cdiv(T * c->heads, RowThreads<D>::kRows), c->device), kThreads, 0,         \
                       static_cast<cudaStream_t>(stream)>>>(s, c->d, d_k, d_v, T, vec)
  WCOMP_KV_DIM(c->dim, CALL);
#undef CALL
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
              a.d_table == a.d_table_out))
    return WCOMP_EINVAL;
  int st = kv_check(c, {a.d_table, a.d_lengths, nullptr, a.B, a.width}, a.B);
  if (st != WCOMP_OK) return st;
  if (int64_t(a.width_out) * kPage >= (int64_t(1) << 31)) return WCOMP_EUNSUPPORTED;
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
  kv4_choose_kernel<<<grid_of(units, c->device), kChoose, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) {
#define CALL(D) kv4_move_kernel<D><<<grid_of(units * int64_t(cdiv(a.keep, kPage)), c->device), kThreads, 0, s>>>(p)
    WCOMP_KV_DIM(c->dim, CALL);
#undef CALL
    e = cudaGetLastError();
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
