// Host-side pieces that the container GEMV (gemv.cu) and the 4-bit and expert
// kernels (q4.cu, moe.cu) share.
#pragma once

#include "wcomp_impl.cuh"

namespace wc {

// The driver's tensor-map encoder, reached through the runtime (no link against
// the driver library); null where it is missing.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encoder();
// A number below kStreams for each of the first kStreams streams that are asked
// for, by the id that the runtime gives a stream and never gives again.  The
// launches on one stream follow one another, so what belongs to its number is used
// by one at a time.  The caller holds its lock.
struct StreamNumbers {
  static constexpr uint32_t kStreams = 1024;
  uint32_t used = 0;
  struct {
    unsigned long long id;
    uint32_t number;  // and 1
  } table[2 * kStreams] = {};
  // -1 when there are more streams
  int of(unsigned long long id) {
    uint64_t i = id % (2 * kStreams);
    while (table[i].number && table[i].id != id) i = (i + 1) % (2 * kStreams);  // half of the table stays empty
    if (!table[i].number) {
      if (used == kStreams) return -1;
      table[i].id = id;
      table[i].number = ++used;
    }
    return int(table[i].number) - 1;
  }
};
// Whether stream s is being captured, and its id where it is not.
inline cudaError_t stream_state(cudaStream_t s, cudaStreamCaptureStatus* capture, cudaGraph_t* graph,
                                unsigned long long* id) {
  const cudaError_t e = cudaStreamGetCaptureInfo(s, capture, nullptr, graph);
  return e != cudaSuccess || *capture != cudaStreamCaptureStatusNone ? e : cudaStreamGetId(s, id);
}
// The expert and 4-bit kernels' error word on device `dev`, null before their
// first use (q4.cu).
uint32_t* work_error_word(int dev);
// Debug builds: which test hooks the launches of q4.cu and moe.cu follow.
cudaError_t debug_hooks_q4(uint32_t bits);
cudaError_t debug_hooks_moe(uint32_t bits);

}  // namespace wc
