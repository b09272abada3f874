/*
 * wcomp.h - lossless BF16 weight coding (byte-split and K15) with a standalone
 * decode and a fused decode-GEMV, for NVIDIA GB300 (sm_103a).
 *
 * The method.  "Prueba de GLM-5.2 reduce la memoria BF16 en casi un 25%"
 * (forgeeks.dev), section "Cómo funciona la compresión": a BF16 weight is
 * 1 sign, 8 exponent and 7 mantissa bits; trained weights reuse a narrow set
 * of sign+exponent symbols.
 *   - byte-split: the high byte (sign + exponent bits 7..1) becomes a 4-bit
 *     code into a per-tensor 15-entry dictionary, code 15 meaning "escape";
 *     escaped high bytes are kept exactly in a (position, byte) stream and
 *     the low byte is stored unchanged (12.005 bits/weight on the pages'
 *     checkpoint, every tensor bit-exact);
 *   - K15: the 9-bit sign+exponent symbol becomes a 4-bit code into a
 *     15-entry table with the same escape rule; the 7-bit mantissa is stored
 *     unchanged (11.173 bits/weight with all overhead on the pages' checkpoint).
 * "Compresión de pesos LLM sin pérdida vs 8-bit GGUF" (wavect.io), section
 * "¿Qué significa “sin pérdida” para los pesos de un LLM?": lossless means the
 * round trip rebuilds every bit; a GPU may keep the weights encoded and rebuild
 * exact BF16 in registers for the matrix product.  Section "Qué queda por
 * demostrar" of the forgeeks page names the open step this library builds: a
 * GEMV that rebuilds the weights in registers and applies the sparse escape
 * correction in the same kernel.
 *
 * Conventions for every entry point below.
 *   - Weights and activations are BF16 bit patterns passed as 16-bit words;
 *     the codec never does float arithmetic on weights, so NaN, Inf, -0 and
 *     subnormals round-trip.
 *   - A weight tensor is W[N, K], row-major (y = x W^T).  n = N * K must be
 *     in [1, 2^32); otherwise WCOMP_EUNSUPPORTED.
 *   - Pointers named d_* are device pointers on the current CUDA device and
 *     are owned by the caller.  `stream` is a cudaStream_t passed as void*
 *     (NULL = the legacy default stream).  Calls are stream-ordered and
 *     asynchronous unless stated otherwise.
 *   - Every call returns a wcomp_status and never aborts; CUDA errors are
 *     WCOMP_ECUDA.  A failed call leaves its outputs unspecified and frees
 *     what it allocated.
 *   - Containers are opaque, owned by the library, and released with
 *     wcomp_free.  A container lives on the device that was current when it
 *     was made.  Container memory comes from a stream-ordered memory pool the
 *     library creates per device; freed blocks stay in that pool for reuse
 *     until the process exits.
 */
#ifndef WCOMP_H
#define WCOMP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define WCOMP_VERSION 1

#if defined(__GNUC__)
#define WCOMP_API __attribute__((visibility("default")))
#else
#define WCOMP_API
#endif

typedef enum { WCOMP_BYTESPLIT = 0, WCOMP_K15 = 1 } wcomp_scheme;

typedef enum {
  WCOMP_OK = 0,
  WCOMP_EINVAL = -1,        /* bad argument (null pointer, size, scheme, B) */
  WCOMP_ENOMEM = -2,        /* device or host allocation failed */
  WCOMP_ECORRUPT = -3,      /* serialized container failed validation */
  WCOMP_ECUDA = -4,         /* a CUDA runtime call failed */
  WCOMP_EUNSUPPORTED = -5,  /* size outside the supported range */
  WCOMP_ETIMEOUT = -6,      /* a kernel's bounded wait on its own copies ran out */
  WCOMP_EINTERNAL = -7,     /* an internal consistency check failed; no result was returned */
  WCOMP_EBOUNDS = -8        /* a debug build's index check failed inside a kernel (the access was skipped) */
} wcomp_status;

typedef struct wcomp_container wcomp_container;

/* Description of a container (filled by wcomp_info). */
typedef struct {
  int32_t scheme;            /* wcomp_scheme */
  int32_t version;           /* container format version */
  int64_t N, K, n;           /* shape and element count */
  uint64_t n_escapes;        /* E: elements whose symbol is not in the table */
  uint32_t tile_elems;       /* granule of the tile escape index (8192) */
  uint32_t n_tiles;
  uint16_t table[15];        /* the 15 symbols, most frequent first */
  uint16_t pad_;
  uint64_t bytes_codes;      /* 4-bit code stream */
  uint64_t bytes_raw;        /* raw low bytes (byte-split) or mantissa planes (K15) */
  uint64_t bytes_index;      /* tile and row escape indexes */
  uint64_t bytes_escapes;    /* escape positions and values */
  uint64_t serialized_bytes; /* header + padded payload */
  double entropy_bpw;        /* 4 + raw bits + (E + 15) * symbol bits / n */
  double physical_bpw;       /* 8 * serialized_bytes / n */
  uint64_t serialized_compact_bytes; /* header + padded payload of the compact form */
  double physical_compact_bpw;       /* 8 * serialized_compact_bytes / n */
} wcomp_info_t;

/*
 * Encode one BF16 tensor.
 *   d_w     device, uint16[N*K] row-major BF16 bits (any alignment; 16-byte
 *           aligned input takes the vector path).
 *   scheme  WCOMP_BYTESPLIT or WCOMP_K15.
 *   out     receives a new container (NULL on failure).
 * Steps (all on the GPU): per-tensor symbol histogram (256 or 512 bins),
 * table of the 15 most frequent symbols (count descending, symbol ascending),
 * 4-bit packing of codes and raw bits, per-tile escape counts and their scan,
 * escape compaction in ascending position order, tile and row escape indexes.
 * Waits on `stream` twice: once for the escape count the histogram implies,
 * which sizes the escape stream (the pack and scan kernels keep running
 * meanwhile), and once for the tile scan, whose total must equal that count
 * (else WCOMP_EINTERNAL and no container).  The escape compaction and the row
 * index are still running on `stream` when the call returns.  Output is
 * deterministic and byte-identical to the CPU oracle.
 * Definition: forgeeks page "Prueba de GLM-5.2 reduce la memoria BF16 en casi
 * un 25%", section "Cómo funciona la compresión": the sign+exponent symbol
 * (8 bits for byte-split, 9 for K15) gets a 4-bit code into the tensor's
 * table of 15 symbols, code 15 marks an escape kept exactly, the low byte or
 * 7-bit mantissa is stored as is.
 */
WCOMP_API int wcomp_encode(const uint16_t* d_w, int64_t N, int64_t K, int scheme, void* stream,
                 wcomp_container** out);

/*
 * How wcomp_encode_batched sizes its histogram grid (host-side, no device
 * work; exposed so the sizing can be checked without a GPU).  n[i] is the
 * element count of tensor i of a batch whose tensors are all histogrammed,
 * sms the device's SM count; blocks[i] receives the number of 256-thread
 * blocks tensor i gets.  Thread t of block b counts the 8-element chunks
 * b * 256 + t, b * 256 + t + 256 * blocks[i], ...; the counters are 16-bit
 * halves shared by 8 threads, so no thread may be given more than 1023
 * chunks (8 x 8 x 1023 = 65472 elements per half).  Returns WCOMP_EINVAL for
 * a null pointer, count or sms <= 0, or an n outside [1, 2^32).
 */
WCOMP_API int wcomp_encode_hist_grid(const uint64_t* n, int count, int sms, uint32_t* blocks);

/*
 * Encode `count` tensors in one pass: tensor i is W_i[N[i], K[i]] at d_w[i],
 * coded with schemes[i]; out[i] receives its container.  The same steps as
 * wcomp_encode run as batched launches over all tensors, with the same two
 * waits on `stream` for the whole batch (escape counts, then the scan check).
 * The batch's containers share two pool blocks (one for their code, raw and
 * index sections, one for their escape streams); each container is still
 * released on its own with wcomp_free, and a block returns to the pool with
 * the last container that uses it.  On failure every out[i] is NULL.
 * Definition: as wcomp_encode (forgeeks page, "Cómo funciona la compresión";
 * one table per tensor).
 */
WCOMP_API int wcomp_encode_batched(const uint16_t* const* d_w, const int64_t* N, const int64_t* K,
                                   const int* schemes, int count, void* stream, wcomp_container** out);

/*
 * Decode a container to exact BF16 bits.
 *   d_out   device, uint16[N*K]; the caller's buffer.
 * The code stream is expanded through the 15-entry table, joined with the raw
 * bits, and escaped elements are patched from the escape stream.
 * Definition: forgeeks page, "Cómo funciona la compresión" (byte-split
 * reconstruction of the high byte; K15 symbol + mantissa).
 */
WCOMP_API int wcomp_decode(const wcomp_container* c, uint16_t* d_out, void* stream);

/*
 * Fused decode-GEMV:  y[b, r] = sum_k x[b, k] * W[r, k]  for b < B, r < N.
 *   d_x     device, uint16[B*K] BF16 bits, row-major, contiguous.
 *   B       batch, 1 <= B <= 16.
 *   d_y     device, float[B*N], row-major; overwritten.
 * W is rebuilt in registers from the codes and raw bits; escaped weights are
 * corrected inside the same kernel (y += x * (w_true - w_placeholder)).
 * Products run on the tensor cores (BF16 MMAs with fp32 accumulation); the
 * summation order is fixed (no atomics), so repeated calls give identical
 * bits.  Shapes with K % 32 != 0 (K15: K % 128 != 0) or an x that is not
 * 16-byte aligned take a slower element-by-element path with the same result
 * contract.
 * Memory: the work counters live in a device buffer the library allocates
 * with cudaMalloc on first use per device (0.5 MB): a pair for each of the
 * first 1024 streams, and 65536 that captured calls (and calls on further
 * streams) take in turn, so that calls on different streams and graphs may run
 * next to one another (a graph next to one captured 65536 calls later may not).
 * A K15 container at B >= 3 also takes a transposed copy of x (K * 4..16 * 2
 * bytes) from the library's stream-ordered pool for the duration of the call.
 * wcomp_gemv_noalloc allocates nothing.
 * Errors found on the device (a copy that never completed) do not fail the
 * call: the kernel records them and stops waiting; wcomp_device_check
 * reports them.
 * Definition: forgeeks page, "Qué queda por demostrar" (GEMV on codes rebuilt
 * in registers, escape correction); wavect page on rebuilding exact BF16 in
 * registers for the matmul.
 */
WCOMP_API int wcomp_gemv(const wcomp_container* c, const uint16_t* d_x, int B, float* d_y, void* stream);

/*
 * wcomp_gemv without any allocation.  The method on the pages has no
 * counterpart to this entry point; it exists for callers that cannot let the
 * library allocate device memory: a serving loop that fixed its memory budget
 * up front, or code that must not meet the implicit device synchronisation a
 * first cudaMalloc or any cudaFree can bring.  wcomp_gemv takes its work
 * counters from a buffer it allocates on first use; this variant keeps them
 * in a 256-byte static device array inside the library instead, which every
 * GPU that loads the library holds until the process exits.
 *   Arguments and results are those of wcomp_gemv.
 *   The first call on a device looks up the array's device address (a
 *   host-side runtime query, no allocation); make that first call before any
 *   stream capture.
 *   Every call shares the one array and zeroes its counters in stream order
 *   before the kernel starts: calls whose kernels overlap on the GPU (on
 *   different streams) race and must be ordered by the caller.
 *   A call covers at most 2^31 - 2^20 rows (N); larger N returns
 *   WCOMP_EUNSUPPORTED.  No cudaMalloc, cudaFree or other allocating routine
 *   is called.
 */
WCOMP_API int wcomp_gemv_noalloc(const wcomp_container* c, const uint16_t* d_x, int B, float* d_y, void* stream);

/*
 * Plain BF16 GEMV over an uncompressed W[N, K] with the same contract as
 * wcomp_gemv; the comparison kernel for the fused path ("0.733x the BF16 GEMV
 * time", forgeeks page, "Qué queda por demostrar").
 */
WCOMP_API int wcomp_gemv_bf16(const uint16_t* d_w, int64_t N, int64_t K, const uint16_t* d_x, int B,
                    float* d_y, void* stream);

/*
 * Batched plain BF16 GEMV: tensor i is W_i[N[i], K[i]] at d_w[i] with input
 * d_x[i] (B x K[i]) and output d_y[i] (B x N[i]); host arrays of length count.
 * The same launch structure as wcomp_gemv_batched, so the two compare like
 * for like.
 */
WCOMP_API int wcomp_gemv_bf16_batched(const uint16_t* const* d_w, const int64_t* N, const int64_t* K,
                                      const uint16_t* const* d_x, int B, float* const* d_y, int count,
                                      void* stream);

/*
 * Batched forms: one launch over `count` containers (any mix of schemes and
 * shapes).  Arrays are host arrays of length count; every d_outs[i] /
 * d_x[i] / d_y[i] is a device buffer sized for containers[i].  All
 * containers must live on the current device.  count may be any positive
 * number (large batches are split into several launches).
 */
WCOMP_API int wcomp_decode_batched(const wcomp_container* const* containers, uint16_t* const* d_outs,
                         int count, void* stream);
WCOMP_API int wcomp_gemv_batched(const wcomp_container* const* containers, const uint16_t* const* d_x,
                       int B, float* const* d_y, int count, void* stream);

/*
 * Report and clear the device error words of the current device (the one
 * wcomp_gemv and the batched GEMVs use, the one in wcomp_gemv_noalloc's
 * static array, and the one of wcomp_q4_gemv and wcomp_moe).  A kernel whose
 * bounded wait on its own tensor copies, or on its other thread blocks, runs
 * out records it there and finishes without waiting instead of hanging; its
 * outputs are then undefined.  Those of other and later calls are not touched, by
 * it or by this check, which may be made while others run.  In a debug build (compiled with WCOMP_DEBUG=1)
 * the kernels on containers and plain weights also check their indexes before
 * memory accesses, skip an access that fails and record it.  Synchronizes
 * `stream`.
 * Returns WCOMP_OK, WCOMP_ETIMEOUT or WCOMP_EBOUNDS.
 */
WCOMP_API int wcomp_device_check(void* stream);

/*
 * Test hooks for the bounded waits, in debug builds only (compiled with
 * WCOMP_DEBUG=1).  While `on` has bit 0 set, every warp of a GEMV launch (fused,
 * plain or 4-bit) or of wcomp_moe (but for BF16 experts that no tensor map
 * takes) leaves the first of its tensor copies unissued but still waits for it:
 * the wait runs out after about a second, the warp stops copying and waiting,
 * lets the copies it has in flight land and finishes, and wcomp_device_check
 * then reports WCOMP_ETIMEOUT.  With bit 1 set, the first thread block of
 * wcomp_moe comes to its first grid barrier half a second after the others gave
 * up on it.  The outputs of such a launch are undefined; the context stays
 * usable.  Applies to the current device and synchronizes it.  Release builds do
 * nothing and return WCOMP_EUNSUPPORTED.  (Library housekeeping; the pages
 * define no counterpart.)
 */
WCOMP_API int wcomp_debug_skip_first_copy(int on);

/*
 * Describe a container (host-side, no device work): shape, table, section
 * sizes, and the bits/weight accounting of forgeeks page "Prueba de GLM-5.2
 * reduce la memoria BF16 en casi un 25%", section "Cómo funciona la
 * compresión" (a 4-bit code plus 8 raw bits for byte-split or 7 for K15 per
 * weight, plus each escape and each table entry at its symbol width), next to
 * the physical bits/weight of both serialized forms.  Returns WCOMP_EINVAL
 * for a NULL argument.
 */
WCOMP_API int wcomp_info(const wcomp_container* c, wcomp_info_t* info);

/*
 * Serialize to a host buffer: a 96-byte header (magic "WCMP", version,
 * scheme, N, K, E, tile size, table, payload length, CRC-32 of the payload,
 * CRC-32 of the header) followed by the payload sections, each padded to 32
 * bytes.  With host_buf == NULL only *len is set.  Returns WCOMP_EINVAL if
 * cap is too small.  Synchronizes `stream`.  The pages fix no file format;
 * this one stores every section the device container holds, so that
 * wcomp_deserialize rebuilds it without recomputation, and carries checksums
 * for the corruption checks of wavect page "Compresión de pesos LLM sin
 * pérdida vs 8-bit GGUF", section "Un piloto de producción de 14 días".
 */
WCOMP_API int wcomp_serialize(const wcomp_container* c, void* host_buf, uint64_t cap, uint64_t* len,
                    void* stream);

/*
 * Serialize to the compact form (format version 2): the same header, then
 * the code stream, the raw bytes (byte-split) or the three K15 mantissa
 * planes, one little-endian uint16 escape count per 8192-element tile, and
 * the escape symbols in ascending position order (byte-split: one byte, the
 * high byte; K15: the 9-bit sign+exponent symbol, packed least significant
 * bit first so that symbol r occupies stream bits 9r .. 9r+8).  Positions,
 * the row index and the K15 escape mantissas are implied (by the codes 15
 * and the planes), so the physical size tracks the bits/weight accounting of
 * forgeeks page "Prueba de GLM-5.2 reduce la memoria BF16 en casi un 25%",
 * section "Cómo funciona la compresión", which counts each escape at its
 * symbol width.  Sections are padded to 32 bytes with zeros.  With host_buf
 * == NULL only *len is set.  Returns WCOMP_EINVAL if cap is too small.
 * Synchronizes `stream`.
 */
WCOMP_API int wcomp_serialize_compact(const wcomp_container* c, void* host_buf, uint64_t cap, uint64_t* len,
                                      void* stream);

/*
 * Rebuild a container from serialized bytes (host buffer), either form.
 * Version 1: the header, both checksums, the section sizes, the escape
 * positions (strictly ascending, below n), both escape indexes and the
 * agreement between escape codes and positions are validated on the host.
 * Version 2 (compact): the header, both checksums and the section sizes are
 * validated, the positions are rebuilt from the codes 15 and must number E,
 * and every tile's escape count must match.  Nothing is copied to the device
 * unless every check passes; any mismatch returns WCOMP_ECORRUPT ("inject
 * corruption" and "validate hashes", wavect page, "Un piloto de producción
 * de 14 días").  Both forms give the same device container.  Synchronizes
 * `stream`.
 */
WCOMP_API int wcomp_deserialize(const void* host_buf, uint64_t len, void* stream, wcomp_container** out);

/*
 * Release a container.  The device memory is returned in stream order on
 * `stream`: work queued earlier on that stream may still use it.  Containers
 * made by one wcomp_encode_batched call share their blocks, which return to
 * the pool on the stream of the last wcomp_free among them: a caller that
 * frees them on different streams orders those streams first.  NULL is a
 * no-op.  (Library housekeeping; the pages define no counterpart.)
 */
WCOMP_API void wcomp_free(wcomp_container* c, void* stream);

/* ------------------------------------------------------------------------
 * Weights in 4 bits with group scales.
 *
 * The lossy sibling of the containers above for callers who can spend the
 * exactness: 4.125 to 4.5 bits per weight instead of 11 to 12, on the same
 * streaming product.  (The pages describe lossless coding only; these entry
 * points have no counterpart there.)
 *
 *   - A weight is M matrices W[N, K], row-major (M = 1 for a plain weight, the
 *     number of experts for wcomp_moe).  Groups are `group` (32, 64 or 128)
 *     consecutive columns of one row, the last one cut off at K.
 *   - A group holds a BF16 scale s and a 4-bit code c (0..15) per weight, which
 *     stands for (c - 8) * s.
 *   - Limits: M, N and K below 2^31, M * ceil(N / 32) below 2^31; beyond them
 *     WCOMP_EUNSUPPORTED.
 *   - A wcomp_q4 is immutable, owned by the library, lives on the device that
 *     was current when it was made (calls with it on another device return
 *     WCOMP_EINVAL), takes its memory from the library's stream-ordered pool,
 *     and is released with wcomp_q4_free.
 * ------------------------------------------------------------------------ */
typedef struct wcomp_q4 wcomp_q4;

typedef struct {
  int64_t M, N, K;
  int32_t group;
  int32_t pad_;
  /* device memory: M * ceil(N / 32) * ceil(K / 256) blocks of 32 rows x 256
     columns, each 4096 bytes of codes and 16384 / group bytes of scales */
  uint64_t bytes;
} wcomp_q4_info_t;

/*
 * Quantise BF16 weights d_w, uint16[M*N*K] (any alignment; 16-byte aligned
 * with K % 8 == 0 takes the vector path).  Per group s = bf16(max |w| / 7),
 * c = clamp(rint(w / s), -7, 7) + 8 with ties to even; s = 0 (zero weights,
 * or a scale that underflows) gives codes 8.  A group that holds an infinity
 * or a NaN gets s = NaN, so what is computed from it is NaN.  Asynchronous.
 */
WCOMP_API int wcomp_q4_encode(const uint16_t* d_w, int64_t M, int64_t N, int64_t K, int group, void* stream,
                              wcomp_q4** out);

/*
 * Take weights that were quantised elsewhere: d_codes uint8[M*N, ceil(K/2)]
 * (column 2j in the low nibble of byte j, 2j + 1 in the high one) and d_scales
 * BF16 bits [M*N, ceil(K/group)].  Every code and any scale is accepted.  The
 * inputs are copied; they may be released in stream order after the call.
 * wcomp_q4_unpack writes the same two arrays (the unused nibble of an odd K's
 * last byte reads 8).
 */
WCOMP_API int wcomp_q4_pack(const uint8_t* d_codes, const uint16_t* d_scales, int64_t M, int64_t N, int64_t K,
                            int group, void* stream, wcomp_q4** out);
WCOMP_API int wcomp_q4_unpack(const wcomp_q4* c, uint8_t* d_codes, uint16_t* d_scales, void* stream);

/*
 * Read back: d_out, uint16[M*N*K], receives (c - 8) * s in BF16, the exact
 * product rounded once to nearest even.
 */
WCOMP_API int wcomp_q4_decode(const wcomp_q4* c, uint16_t* d_out, void* stream);

/*
 * y[b, r] = sum_k x[b, k] * (c[r, k] - 8) * s[r, group of k], b < B, r < N, for
 * a weight of one matrix (M == 1).  d_x uint16[B*K] BF16 bits, 1 <= B <= 16;
 * d_y float[B*N], overwritten.  Any alignment of d_x.
 * Numbers: x is taken in blocks of 128 columns as fp16 under the power of two
 * that its largest magnitude asks for.  A BF16 value keeps all its bits down to
 * 2^-31 of that; smaller ones err by at most 2^-39 of it.  Products with c - 8
 * are then exact and summed in fp32 on the tensor cores; a group's sum enters
 * the fp32 result under scale times power of two, which is exact.  So a scale
 * may be large where x is small, and small where x is large: what is asked is
 * that scale times the largest magnitude of x in its 128 columns be below 2^128;
 * where that is below 2^-128 a group errs by up to 2^-125.  Infinities and NaN of
 * x stay in their row of x and follow the definition; an infinite or NaN scale
 * makes its row of the weight infinite or NaN.  The order of the sums is fixed:
 * repeated calls give identical bits.
 * Memory: that form of x and, where rows are split over thread blocks, their
 * parts come from the library's stream-ordered pool for the duration of the
 * call.  The device's error word is allocated with cudaMalloc on first use: make
 * the first call before any stream capture.
 */
WCOMP_API int wcomp_q4_gemv(const wcomp_q4* c, const uint16_t* d_x, int B, float* d_y, void* stream);

/* Describe a weight (host-side, no device work). */
WCOMP_API int wcomp_q4_info(const wcomp_q4* c, wcomp_q4_info_t* info);

/*
 * Release a weight: work queued earlier on `stream` may still use it.  NULL is
 * a no-op.
 */
WCOMP_API void wcomp_q4_free(wcomp_q4* c, void* stream);

/* ------------------------------------------------------------------------
 * A mixture-of-experts layer for a few tokens.
 * ------------------------------------------------------------------------ */
typedef enum { WCOMP_MOE_SOFTMAX = 0, WCOMP_MOE_SIGMOID = 1 } wcomp_moe_scoring;

typedef struct {
  /* x[T, H] and router[E, H], BF16 bits, row-major; bias[E] fp32 or NULL */
  const uint16_t* d_x;
  const uint16_t* d_router;
  const float* d_bias;
  /* experts, all three as BF16 rows (gate, up: [E, F, H]; down: [E, H, F]) or
     all three in 4 bits with one group size (M = E); the other form NULL */
  const uint16_t* d_gate;
  const uint16_t* d_up;
  const uint16_t* d_down;
  const wcomp_q4* q4_gate;
  const wcomp_q4* q4_up;
  const wcomp_q4* q4_down;
  /* y[T, H] BF16 bits, overwritten; may be x itself */
  uint16_t* d_y;
  /* optional outputs, [T, top_k]: the experts in the order of their choice and
     the weights they got */
  int32_t* d_ids;
  float* d_weights;
  int64_t H, F;
  int32_t T, E, top_k;
  int32_t scoring;      /* wcomp_moe_scoring */
  int32_t renormalize;  /* divide the chosen scores by their sum (at least 1e-20) */
  float factor;         /* multiplies the weights */
} wcomp_moe_args;

/*
 * One layer for T tokens, 1 <= T <= 16, in one kernel:
 *   l[t, e] = x[t] . router[e];  score = softmax over e, or sigmoid, of l;
 *   the top_k experts of largest score + bias are chosen (bias only steers the
 *   choice; ties go to the lowest index; a NaN ranks below everything; an
 *   expert whose bias is -inf is chosen only when no other is left);
 *   weight[t, j] = factor * score, divided by the chosen scores' sum if
 *   renormalize;
 *   y[t] = sum_j weight[t, j] * down_j (silu(gate_j x[t]) * (up_j x[t])).
 * Sums and scores are in fp32 (experts whose scores are 0 there, from logits of
 * 104 under the largest or, for sigmoid, under zero on, count as ties).  The hidden
 * values between the products are held as two BF16 parts (BF16 experts: 16
 * significant bits) or in fp16 under a power of two for each 32 of them (4-bit
 * experts: 11 bits, an eighth of a step of the result; x as in wcomp_q4_gemv).  y is
 * rounded once.  The order of the sums is fixed: repeated calls give identical bits.
 * 1 <= top_k <= min(E, 16), E <= 1024, H and F at most 2^24 (beyond:
 * WCOMP_EUNSUPPORTED).  Any alignment and widths; BF16 experts with H % 8 == 0,
 * F % 8 == 0 and 16-byte aligned weights are copied in boxes through tensor
 * maps, others in 4-byte words, with the same results to the order of a sum.
 * Experts that no token chose are not read.
 * The kernel is launched cooperatively (its thread blocks meet at two grid
 * barriers).  Waits are bounded: if one runs out, the kernel finishes with
 * undefined outputs and wcomp_device_check reports WCOMP_ETIMEOUT.
 * Memory: logits, hidden values, parts of sums and (unless x can be read as it
 * is) a copy of x come from the library's stream-ordered pool for the duration
 * of the call.  The counters of the barriers are allocated with cudaMalloc on
 * first use (25 MB; make the first call before any stream capture): a set for each
 * of the first 1024 streams that the device's calls are made on, one for good for
 * each of the first 1024 captured calls, and one for each of 4096 others while
 * their graphs are there (which costs a graph's launch 2.3 us and 0.14 us a call),
 * so that calls on different streams and graphs may run next to one another.
 * Calls beyond these clear counters of their own, which takes them 4 us longer.
 */
WCOMP_API int wcomp_moe(const wcomp_moe_args* args, void* stream);

/* Human-readable text for a status code (static string). */
WCOMP_API const char* wcomp_strerror(int status);

/* WCOMP_VERSION of the library that was loaded. */
WCOMP_API int wcomp_version(void);

/*
 * Number of CUDA kernels this library has launched in the calling process
 * (all devices, all threads).  Host-side counter, no device work; used to
 * report how many of the library's own kernels a timed region ran.
 */
WCOMP_API uint64_t wcomp_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* WCOMP_H */
