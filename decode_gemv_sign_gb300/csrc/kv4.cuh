// The 4-bit key/value cache: its layout, and where a call's rows stand in it.
// Shared by the calls that write and read it (kv4.cu) and by the attention over
// it (kv4_attend.cu).
#pragma once

#include "pairs.cuh"
#include "tile.cuh"

struct wcomp_kv4 {
  int64_t pages = 0;
  int heads = 0, dim = 0;
  int device = 0;
  uint8_t* d = nullptr;
};

namespace wc {

constexpr int kPage = 64;       // tokens of a page
constexpr int kKvGroup = 32;    // columns that share a scale

// A page holds one block per head, its first half the keys and its second the
// values: 64 rows of codes (dim / 2 bytes each) and the scales [dim / 32][64],
// BF16.  A block is one bulk copy of the attention and a multiple of 128 bytes; a
// row is made of whole 16-byte pieces, so that a token can be written and moved
// by itself.
//
// In a key row the 8 columns 32 g + 8 q .. + 7 are the word q * G + g (G = dim /
// 32; column i of them in bits 4 i .. 4 i + 3): lane q of a quad of the MMA finds its
// columns of every group in consecutive words.  In a value row word r * G / 2 + a
// holds the columns 64 a + 4 r .. + 3 in its low and 64 a + 32 + 4 r .. + 3 in its
// high half: lane r of the MMA's eight rows finds its columns of every group in
// consecutive words.
//
// The attention's lane (r, q) reads key rows of the tokens 8 i + r and value rows of
// 8 i + 2 q and 8 i + 2 q + 1; a token's row is swizzled so that both spread over
// all banks, and the scales of the tokens r, 8 + r, 16 + r, ... lie together.
template <int D>
struct Kv {
  static constexpr int G = D / kKvGroup;
  static constexpr uint32_t kRow = D / 2;
  static constexpr uint32_t kCodes = kPage * kRow;
  static constexpr uint32_t kHalf = kCodes + G * kPage * 2;
  static constexpr uint32_t kBlock = 2 * kHalf;
  // From the start of the keys or the values: byte b of token t's row, and its
  // scale of group g.
  static __host__ __device__ __forceinline__ uint32_t at(uint32_t t, uint32_t b) {
    const uint32_t turn = D == 64 ? (t >> 2) & 1 : (t >> 1) & 3;
    return (t * kRow + b) ^ (turn << 5) ^ (D == 256 ? (t & 1) << 4 : 0);
  }
  static __host__ __device__ __forceinline__ uint32_t scale(uint32_t t, uint32_t g) {
    return kCodes + 2 * (g * kPage + (t & 7) * 8 + (t >> 3));
  }
};

// The rows of a call (wcomp_kv4_seqs) on the device.
struct KvSeqs {
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* starts;  // or null
  int B, width;
  uint32_t pages, heads;  // of the cache
  uint32_t* err;
};

__device__ __forceinline__ void kv_bad(uint32_t* err) { atomicOr(err, kErrBounds); }

// Tokens that sequence b holds.
__device__ __forceinline__ int kv_length(const KvSeqs& s, int b) {
  const int n = s.lengths[b];
  if (n <= s.width * kPage) return n < 0 ? 0 : n;
  kv_bad(s.err);
  return s.width * kPage;
}
// Page number `at` of sequence b, -1 if there is no such page.
__device__ __forceinline__ int kv_page(const KvSeqs& s, int b, int at) {
  const int p = s.table[int64_t(b) * s.width + at];
  if (uint32_t(p) < s.pages) return p;
  kv_bad(s.err);
  return -1;
}
// Sequence of row i, or -1.
__device__ __forceinline__ int kv_sequence(const KvSeqs& s, int64_t i) {
  if (!s.starts) return i < s.B ? int(i) : -1;
  if (i < s.starts[0] || i >= s.starts[s.B]) return -1;
  int lo = 0, hi = s.B;  // starts[lo] <= i < starts[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.starts[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}
// Position of row i of sequence b, which holds n tokens; below 0: none.
__device__ __forceinline__ int64_t kv_position(const KvSeqs& s, int b, int64_t i, int n) {
  return s.starts ? int64_t(n) - (s.starts[b + 1] - i) : int64_t(n) - 1;
}

// Report starts that descend, are negative or pass the call's T rows: thread `at` of `threads`.
__device__ __forceinline__ void kv_check_starts(const KvSeqs& s, int64_t T, uint32_t at, uint32_t threads) {
  if (!s.starts) return;
#pragma unroll 1
  for (int64_t b = at; b < s.B; b += threads)
    if (s.starts[b] < 0 || s.starts[b + 1] < s.starts[b] || s.starts[b + 1] > T) kv_bad(s.err);
}

// Checks of a call's sequences on the host.
int kv_check(const wcomp_kv4* c, const wcomp_kv4_seqs& s, int64_t T);
int kv_seqs(const wcomp_kv4* c, const wcomp_kv4_seqs& s, KvSeqs* out);

}  // namespace wc
