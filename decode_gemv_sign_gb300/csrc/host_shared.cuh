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
// The expert and 4-bit kernels' error word on device `dev`, null before their
// first use (q4.cu).
uint32_t* work_error_word(int dev);
// Debug builds: which test hooks the launches of q4.cu and moe.cu follow.
cudaError_t debug_hooks_q4(uint32_t bits);
cudaError_t debug_hooks_moe(uint32_t bits);

}  // namespace wc
