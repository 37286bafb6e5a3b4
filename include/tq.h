/*
 * tq.h -- C ABI of libtq: the TQ4_1S weight codec and its fused dequant-GEMV
 * for NVIDIA B200 (sm_100a).
 *
 * Source of the method: the web page titled "企业官网建设流程全解析"
 * (hotelren.com/news/5458160; below "TQ page"), which describes TQ4_1S weight
 * compression: paragraph 格式原理 items 1-3 (sign flip + 32-point Walsh-Hadamard
 * rotation per block, nearest of 16 Lloyd-Max N(0,1) centroids, separate
 * scales d0/d1 for elements 0-15 and 16-31), the paragraph after them (16
 * centroids, nibble packing, no correction term; the reference dequantiser
 * inverse-rotates and rescales) and section 解码速度：分硬件汇总 (decode
 * pre-rotates the activation once, so dequantisation becomes centroid
 * lookup times scale).
 *
 * ---------------------------------------------------------------------------
 * Conventions shared by every entry point
 * ---------------------------------------------------------------------------
 *  - W is N x K (out_features x in_features), row-major; y = W x.  Blocks of
 *    32 run along K; K must be a positive multiple of 32.
 *  - Pointers named codes/scales/w/x/y/workspace/xrot are DEVICE pointers on
 *    the current CUDA device; the caller owns and allocates all of them.
 *    The library allocates no memory and keeps no state beyond constant
 *    tables.  stream is a cudaStream_t (NULL = legacy default stream).
 *  - Calls are asynchronous on `stream` and never synchronise.  Argument
 *    errors are detected on the host before any launch and nothing is
 *    launched; a launch failure returns TQ_ERR_CUDA.
 *  - n == 0 or m == 0 is an empty problem: TQ_OK, nothing launched.
 *  - All results are deterministic run to run (no floating-point atomics).
 *
 * Packed format (5.0 bits per weight when N % 16 == 0 and K % 128 == 0):
 *  - code: 4 bits; bit 3 = sign (1 = negative), bits 0-2 = magnitude rank
 *    0..7 into the eight positive Lloyd-Max centroids.
 *  - superblock = four consecutive 32-element blocks of one row (128
 *    columns); NSB = ceil(K/128).  Rows are grouped in tiles of 16
 *    (T = ceil(N/16)).  A unit = (tile, superblock) is stored contiguously and
 *    units are tile-major, so the fused kernel streams 1024 + 256 contiguous
 *    bytes per unit.  Blocks past K/32 and rows past N are zero.
 *  - codes plane: uint8 [T][NSB][16 rows][64].  Within a row's 64 bytes,
 *    logical byte L (0..15) of block j (0..3) holds the codes of elements 2L
 *    (low nibble) and 2L+1 (high nibble) and is stored at byte
 *    16*(L%4) + 4*j + L/4.
 *  - scales plane: uint16 [T][NSB][16 rows][4 blocks][2], IEEE fp16 bit
 *    patterns d0, d1: d_h = fp16(sqrt(mean of the 16 squared rotated values)).
 *  - rotation: y = H (s .* w) per block, H the unnormalised 32x32 Sylvester
 *    Hadamard matrix; s_k = -1 where bit 31 of hash(k) is set, with
 *    hash(k) = g(k * 0x9E3779B9) and g(h) = ((h ^ h>>16) * 0x85EBCA6B) ^ (...>>13)
 *    on 32-bit words, k = global column index (same for every row).
 *  - dequantisation: w~ = s .* (H c) / 32, c_e = +-M[mag_e] * d_h(e).
 */
#ifndef TQ_H_
#define TQ_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define TQ_API __attribute__((visibility("default")))
#else
#define TQ_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TQ_OK = 0,
    TQ_ERR_INVALID_ARG = 1, /* null pointer, bad leading dimension, negative size */
    TQ_ERR_SHAPE = 2,       /* k <= 0, k % 32 != 0, or a size above the supported maximum */
    TQ_ERR_ALIGNMENT = 3,   /* a pointer or leading dimension breaks the alignment rule */
    TQ_ERR_DTYPE = 4,       /* unknown tq_dtype value */
    TQ_ERR_WORKSPACE = 5,   /* workspace null or smaller than the *_workspace_bytes query */
    TQ_ERR_CUDA = 6,        /* a CUDA runtime call or launch failed */
    TQ_ERR_UNSUPPORTED = 7, /* valid request that this build does not implement */
    TQ_ERR_TIMEOUT = 8      /* a kernel's bounded wait expired (tq_workspace_status) */
} tq_status;

typedef enum { TQ_F32 = 0, TQ_BF16 = 1, TQ_F16 = 2 } tq_dtype;

/* Largest supported sizes (checked; TQ_ERR_SHAPE above them). */
#define TQ_MAX_N ((int64_t)1 << 30)
#define TQ_MAX_K ((int64_t)1 << 26)
#define TQ_MAX_BATCH 8

/* Human-readable name of a status code (static string, never NULL). */
TQ_API const char *tq_status_string(tq_status s);

/* Bytes of the codes plane / of the scales plane for an N x K matrix
 * (ceil(n/16) * ceil(k/128) * 1024 and ceil(n/16) * ceil(k/128) * 256).
 * 0 for invalid sizes. */
TQ_API size_t tq_codes_bytes(int64_t n, int64_t k);
TQ_API size_t tq_scales_bytes(int64_t n, int64_t k);

/*
 * tq_quantize -- encode W into the packed TQ4_1S planes.
 * TQ page, 格式原理 items 1-3 and the paragraph after them: per 32-block,
 * sign flip + Walsh-Hadamard rotation, two fp16 RMS half-block scales, then
 * for every rotated value y the code sign(y) / #{j : |y| > B_j * d} with the
 * seven Lloyd-Max decision thresholds B_j (ties go to the smaller magnitude,
 * +0 and -0 count as positive).  Every step is IEEE fp32 in a fixed order,
 * so codes and scales are bit-reproducible by a CPU implementation.
 *   w      device, n x k of dtype wt (F32, BF16 or F16), row stride ldw
 *          elements (ldw >= k, ldw % 8 == 0, w 16-byte aligned)
 *   codes  device, tq_codes_bytes(n, k) bytes, 16-byte aligned (written)
 *   scales device, tq_scales_bytes(n, k) bytes, 16-byte aligned (written)
 * Inputs with |w| large enough to overflow fp16 scales (RMS >= 65520) or
 * containing NaN/Inf are outside the contract.
 */
TQ_API tq_status tq_quantize(const void *w, tq_dtype wt, int64_t n, int64_t k, int64_t ldw, uint8_t *codes,
                      uint16_t *scales, void *stream);

/*
 * tq_dequantize -- reconstruct w~ = s .* (H c) / 32 (TQ page, paragraph after
 * 格式原理: inverse rotation and rescale).  fp32 arithmetic, output rounded
 * to ot (nearest-even).
 *   codes, scales  device, as written by tq_quantize for the same n, k
 *   w_out  device, n x k of dtype ot, row stride ldo (ldo >= k, ldo % 8 == 0,
 *          16-byte aligned)
 */
TQ_API tq_status tq_dequantize(const uint8_t *codes, const uint16_t *scales, int64_t n, int64_t k, void *w_out,
                        tq_dtype ot, int64_t ldo, void *stream);

/*
 * tq_dequantize_batch -- tq_dequantize of count (1..TQ_MAX_BATCH) matrices in
 * one launch, every output of dtype ot (e.g. all seven matrices of a layer;
 * one launch has one ramp and one tail instead of seven).  The same argument
 * rules as tq_dequantize per descriptor; descriptors with n == 0 are skipped.
 * Outputs must not overlap one another or any codes/scales.
 */
typedef struct {
    const uint8_t *codes;   /* device, packed planes of an n x k matrix (tq_quantize) */
    const uint16_t *scales;
    int64_t n;              /* >= 0 */
    int64_t k;              /* positive multiple of 32 */
    void *w_out;            /* device, n x k of dtype ot, row stride ldo (ldo >= k, ldo % 8 == 0, 16-byte aligned) */
    int64_t ldo;
} tq_dequant_desc;
TQ_API tq_status tq_dequantize_batch(const tq_dequant_desc *descs, int count, tq_dtype ot, void *stream);

/*
 * Pre-rotated activations (TQ page, 解码速度 section: the activation is
 * rotated once and shared, so the per-weight work is lookup x scale).
 * xrot holds fp16 values H(s .* x)/32 per 32-block, in the order the fused
 * kernel's tensor-core fragments read them: [m][NSB][4 blocks][4][8], where
 * entry [t][q] of a block is element (q/2)*8 + 2t + (q%2).  Padding blocks
 * are zero.  |x| must stay below 65504 (fp16 range).
 */
TQ_API size_t tq_xrot_bytes(int64_t m, int64_t k);

/*
 * tq_prerotate -- xrot = fragment-ordered fp16(H (s .* x) / 32) for each of the
 * m rows of X.
 *   X     device, m x k of dtype xt, row stride ldx (ldx >= k, ldx % 8 == 0,
 *         16-byte aligned)
 *   xrot  device, tq_xrot_bytes(m, k) bytes, 16-byte aligned (written)
 */
TQ_API tq_status tq_prerotate(const void *X, tq_dtype xt, int64_t m, int64_t k, int64_t ldx, uint16_t *xrot,
                       void *stream);

/* Workspace bytes needed by tq_gemm / tq_gemv / tq_gemm_xrot on the CURRENT
 * device for these sizes (the split-K partition depends on its SM count).
 * Layout: a 256-byte header (status word, call tag), the split-K partial
 * sums and the pre-rotated activation.
 *
 * Every call clears the status word and advances the 32-bit call tag before
 * its product; split-K partial sums are stored together with the tag of
 * their call, so words left by earlier calls never match.  A workspace that
 * has never been used holds arbitrary bytes and a stale word could match the
 * first call's tag by chance (probability 2^-32 per word read): zero-fill a
 * new workspace once (later calls need no clearing). */
TQ_API size_t tq_gemm_workspace_bytes(int64_t m, int64_t n, int64_t k);

/*
 * tq_gemm -- Y[i][r] = sum_k w~[r][k] X[i][k] for i < m, r < n, computed as
 * (1/32) sum_blocks sum_halves d * sum_e c_e xrot_e with the activation
 * pre-rotated once per call (TQ page, 解码速度 section).  Centroids and xrot
 * enter the tensor cores as fp16; products accumulate in fp32.
 * Kernels: m <= 8 runs the mma.sync kernel (half-block sums scaled in fp32);
 * m = 9..32 runs the tcgen05 kernel that stages the decoded weights in tensor
 * memory; m > 32 runs the prefill product.  From m = 9 (and for m = 25..32
 * on the mma.sync kernel when a test hook forces it) the centroid enters
 * already multiplied by its half-block scale, fp16(c * d): that product
 * overflows once d exceeds about 23,970 (weights of magnitude around 4,000
 * and up) and becomes an fp16 subnormal, with coarser relative precision,
 * once 0.128 * d falls below 6.1e-5, i.e. d below about 4.8e-4 (weights of
 * RMS below about 1e-4).
 *   X          device, m x k of dtype xt, row stride ldx (as tq_prerotate)
 *   Y          device, m x n of dtype yt (F32, BF16 or F16), row stride ldy
 *              (ldy >= n)
 *   workspace  device, >= tq_gemm_workspace_bytes(m, n, k) bytes, 256-byte
 *              aligned, exclusively owned by this call until it completes
 *              on `stream` (zero-filled once when new, see above; calls
 *              that overlap on the GPU must use different workspaces)
 * m <= 32 runs the skinny kernel in one pass; larger m runs the tensor-core
 * prefill product of tq_gemm_prefill (its workspace is then the size that
 * tq_gemm_workspace_bytes(m, n, k) returns for that m).
 */
TQ_API tq_status tq_gemm(const uint8_t *codes, const uint16_t *scales, int64_t n, int64_t k, const void *X, tq_dtype xt,
                  int64_t m, int64_t ldx, void *Y, tq_dtype yt, int64_t ldy, void *workspace, size_t ws_bytes,
                  void *stream);

/* tq_gemv -- tq_gemm with m = 1 (x: k elements, y: n elements). */
TQ_API tq_status tq_gemv(const uint8_t *codes, const uint16_t *scales, int64_t n, int64_t k, const void *x, tq_dtype xt,
                  void *y, tq_dtype yt, void *workspace, size_t ws_bytes, void *stream);

/*
 * tq_gemm_prefill -- the same product for many activation rows (prefill) on
 * the fifth-generation tensor cores (TQ page, 解码速度 section: rotate the
 * activation once, then every weight is centroid times scale).  X is first
 * pre-rotated into a plain row-major fp16 matrix in the workspace; then each
 * CTA takes 256 weight rows x 256 activation rows: it decodes its weight rows
 * 64 columns at a time into shared memory (centroid x half-block scale, fp16),
 * receives the matching activation columns by TMA, and accumulates
 * tcgen05.mma products (fp16 operands, two fp32 accumulators in tensor
 * memory, one per 128-row half of the weight tile).
 * Compared with tq_gemm's skinny path the weight enters as fp16(c * d), one
 * more rounding per weight (relative 2^-11).  Same operand rules as tq_gemm;
 * any m >= 1 (m <= 16,776,960).  Returns TQ_ERR_UNSUPPORTED if the driver
 * offers no tensor-map encoder.
 *   workspace  >= tq_gemm_prefill_workspace_bytes(m, k) bytes (256-byte
 *              header + m*k fp16), 256-byte aligned
 */
TQ_API size_t tq_gemm_prefill_workspace_bytes(int64_t m, int64_t k);
TQ_API tq_status tq_gemm_prefill(const uint8_t *codes, const uint16_t *scales, int64_t n, int64_t k, const void *X,
                                 tq_dtype xt, int64_t m, int64_t ldx, void *Y, tq_dtype yt, int64_t ldy,
                                 void *workspace, size_t ws_bytes, void *stream);

/*
 * The two steps of tq_gemm_prefill as separate calls, so that one rotated
 * activation serves every matrix that consumes it (e.g. q/k/v in a prefill;
 * TQ page, paragraph 适用前提与边界, the attention tensors share one rotation).
 *
 * tq_prefill_xrot_bytes -- m * k * 2: the plain pre-rotated activation, a
 * row-major m x k fp16 matrix, element [i][c] = fp16(H(s .* x_i)/32) at
 * column c (blocks of 32 along k, in order).
 *
 * tq_prerotate_plain -- writes that matrix for the m rows of X.
 *   X     device, m x k of dtype xt, row stride ldx (as tq_prerotate)
 *   xrot  device, tq_prefill_xrot_bytes(m, k) bytes, 16-byte aligned
 *         (written; read by tensor-memory-accelerator copies afterwards)
 *
 * tq_gemm_prefill_xrot -- the tensor-core product of tq_gemm_prefill over an
 * xrot written by tq_prerotate_plain (same m and k).  The workspace needs
 * only its 256-byte header (>= 256 bytes, 256-byte aligned); a one-thread
 * launch clears its status word first.  Y, yt, ldy as tq_gemm.
 */
TQ_API size_t tq_prefill_xrot_bytes(int64_t m, int64_t k);
TQ_API tq_status tq_prerotate_plain(const void *X, tq_dtype xt, int64_t m, int64_t k, int64_t ldx, uint16_t *xrot,
                                    void *stream);
TQ_API tq_status tq_gemm_prefill_xrot(const uint8_t *codes, const uint16_t *scales, int64_t n, int64_t k,
                                      const uint16_t *xrot, int64_t m, void *Y, tq_dtype yt, int64_t ldy,
                                      void *workspace, size_t ws_bytes, void *stream);

/*
 * tq_gemm_xrot -- the product with an activation already pre-rotated by
 * tq_prerotate (one xrot shared by every matrix that consumes the same
 * input, e.g. q/k/v).  m <= 32.  Same workspace rules as tq_gemm (a
 * one-thread launch on `stream` clears the status word and advances the call
 * tag before the product).
 */
TQ_API tq_status tq_gemm_xrot(const uint8_t *codes, const uint16_t *scales, int64_t n, int64_t k, const uint16_t *xrot,
                       int64_t m, void *Y, tq_dtype yt, int64_t ldy, void *workspace, size_t ws_bytes, void *stream);

/*
 * Several matrices in one launch (TQ page, paragraph 适用前提与边界: the
 * attention tensors of a layer share one in-place rotation, i.e. matrices
 * that consume the same input can share one pre-rotated activation).
 * Every descriptor is one product Y = X w~^T with its own codes/scales;
 * descriptors with the same X pointer, k and ldx share one pre-rotation.
 * One launch pre-rotates every distinct input, one launch computes every
 * product (no per-matrix launch overhead).
 */
typedef struct {
    const uint8_t *codes;   /* device, packed planes of an n x k matrix */
    const uint16_t *scales;
    int64_t n;              /* >= 1 */
    int64_t k;              /* positive multiple of 32 */
    const void *X;          /* device, m x k activations (dtype xt), row stride ldx */
    int64_t ldx;
    void *Y;                /* device, m x n outputs (dtype yt), row stride ldy */
    int64_t ldy;
} tq_gemm_desc;

/* Workspace bytes for tq_gemm_batch on the current device (0 if invalid). */
TQ_API size_t tq_gemm_batch_workspace_bytes(const tq_gemm_desc *descs, int count, int64_t m);

/* tq_gemm_batch -- count (1..TQ_MAX_BATCH) products with m <= 32 activation
 * rows each; the same argument rules as tq_gemm per descriptor. */
TQ_API tq_status tq_gemm_batch(const tq_gemm_desc *descs, int count, int64_t m, tq_dtype xt, tq_dtype yt,
                               void *workspace, size_t ws_bytes, void *stream);

/*
 * tq_workspace_status -- synchronises `stream`, then reports whether the last
 * product that used this workspace hit a bounded wait (TQ_ERR_TIMEOUT: the
 * kernel gave up on a bulk copy after ~1 s, recorded it and returned; its
 * outputs are then incomplete).  clear != 0 resets the flag.  The flag is
 * also reset by the next tq_gemm / tq_gemv / tq_gemm_xrot / tq_gemm_batch
 * on the workspace.
 */
TQ_API tq_status tq_workspace_status(void *workspace, int clear, void *stream);

/*
 * tq_debug_set_flags -- test hook, process-wide, 0 by default.  Bit 0: in
 * later fused-product launches (m <= 32) the first copy of the first warp
 * (mma.sync kernel) or of the first CTA (tensor-memory kernel) is never
 * issued, so its bounded wait expires after ~5 ms and the timeout path runs
 * (status word set, kernel returns normally; no fault, no trap).  Bits 2 and
 * 3: every product with m <= 32 runs on the tensor-memory kernel (bit 2) or
 * on the mma.sync kernel (bit 3) instead of the kernel chosen by m.  Bit 4:
 * in the mma.sync kernel the first warp of every split tile recomputes the
 * later warps' contributions from the packed weights instead of reading
 * them (the path it takes when a contribution does not arrive within 50 us,
 * e.g. because another kernel holds the SMs its CTA needs); the result is
 * bit-identical.  Bit 1:
 * the same for the tensor-core prefill product (tq_gemm_prefill and m > 32):
 * the first CTA never issues its second activation-tile copy (nor counts its
 * bytes), its waits expire after ~5 ms, every tensor-memory column is still
 * released, and the status word is set.  Bit 5: the same for the tcgen05
 * attention kernel (tq_kv_attention): the first tile's first keys are never
 * handed over.  Bit 6: that kernel's last CTA takes its tensor memory for
 * incomplete and reports it.
 */
TQ_API void tq_debug_set_flags(uint32_t flags);

/*
 * tq_gemv_static_scratch -- the GEMV of tq_gemv for callers that cannot
 * allocate device memory (code inside an allocator or memory-pool callback,
 * plugins that only receive an operation's tensors, processes whose device
 * memory is all reserved up front).  The pages this library follows have no
 * counterpart to it: it exists only for such callers.
 *
 * Inputs and outputs are as for tq_gemv (x: k elements, y: n elements, both
 * device memory supplied by the caller); no workspace is passed.  Instead the
 * scratch lives in one fixed device array of TQ_STATIC_SCRATCH_BYTES inside
 * the library, present on every GPU that loads it until the process exits.
 * The call allocates nothing (no cudaMalloc, cudaFree or allocating library
 * routine) and returns TQ_ERR_SHAPE when the problem's scratch,
 * tq_gemm_workspace_bytes(1, n, k), exceeds TQ_STATIC_SCRATCH_BYTES.
 *
 * The first call in a CUDA context looks up the array's device address
 * (cudaGetSymbolAddress) with that context's device current; make that first
 * call before any stream capture.  The address is cached per context (keyed
 * by the driver's unique context id), so after cudaDeviceReset, or from
 * another context on the same device, the next call looks it up again; do
 * that call outside stream capture too.  All calls share the array, and each
 * starts by clearing what must start at zero: calls that overlap on the GPU
 * (other streams, other host threads, without ordering between them) race
 * and give wrong results.  Run them in order on one stream (or order the
 * streams with events), or use tq_gemv.
 *
 * A bounded wait that expires inside this call is recorded in the array's
 * status word like tq_gemv's: read it with tq_static_scratch_status.
 */
#define TQ_STATIC_SCRATCH_BYTES (4u << 20)

TQ_API tq_status tq_gemv_static_scratch(const uint8_t *codes, const uint16_t *scales, int64_t n, int64_t k,
                                        const void *x, tq_dtype xt, void *y, tq_dtype yt, void *stream);

/*
 * tq_static_scratch_status -- tq_workspace_status for the fixed array of
 * tq_gemv_static_scratch in the current context: synchronises `stream`, then
 * returns TQ_ERR_TIMEOUT if the last tq_gemv_static_scratch call on this
 * device gave up a bounded wait (its y is then incomplete), else TQ_OK;
 * clear != 0 resets the flag (the next call also resets it).  Allocates
 * nothing.
 */
TQ_API tq_status tq_static_scratch_status(int clear, void *stream);

/*
 * ---------------------------------------------------------------------------
 * NVFP4 comparison codec
 * ---------------------------------------------------------------------------
 * NVFP4 is named, without a bit recipe, by the llm-compressor page
 * (ai-insight.org/news/11771: NVFP4 checkpoints) and the llama.cpp quantizer
 * page (bittide.aicompass.dev: "NVFP4 weight and input tensor scales").  This
 * library implements the plainest reading of the format, for comparison with
 * TQ4_1S on the same shapes:
 *   g   = amax|W| / (6 * 448)                       fp32, one per tensor
 *   s_b = E4M3(amax_b / (6 * g))                    one per 16 elements
 *   q   = E2M1(w / (value(s_b) * g))                4 bits per element, 0 when
 *                                                   the scale is 0
 *   w~  = value(q) * value(s_b) * g
 * Each quotient and product is one IEEE fp32 operation; both conversions
 * round to nearest-even and saturate (E4M3 at 448, E2M1 at 6); a zero code
 * carries no sign.  No rotation.  4.5 bits per weight.
 *
 * Layout: the codes plane is the TQ4_1S one (tq_codes_bytes; the two
 * 16-element blocks of a 32-column pair take the place of one 32-element
 * block, byte order unchanged: element 2L in the low nibble of logical byte
 * L).  E2M1 code: bit 3 = sign, bits 0-2 = magnitude index into
 * {0, 0.5, 1, 1.5, 2, 3, 4, 6}.  The scales plane is E4M3 bytes
 * [T][NSB][16 rows][8 blocks of 16] (tq_nvfp4_scales_bytes).  The tensor
 * block is TQ_NVFP4_TENSOR_BYTES of device memory: float g at offset 0, the
 * fp32 amax|W| at offset 4, the rest reserved.
 */
#define TQ_NVFP4_TENSOR_BYTES 16

/* ceil(n/16) * ceil(k/128) * 128 bytes; 0 for invalid sizes. */
TQ_API size_t tq_nvfp4_scales_bytes(int64_t n, int64_t k);

/*
 * tq_nvfp4_quantize -- encode W (n x k, dtype wt, row stride ldw; the operand
 * rules of tq_quantize) into codes (tq_codes_bytes), scales
 * (tq_nvfp4_scales_bytes) and the tensor block (TQ_NVFP4_TENSOR_BYTES); all
 * device, 16-byte aligned, written.  Three operations on `stream`: a memset of
 * the amax word, a reduction of amax|W|, the encode.  NaN/Inf inputs are
 * outside the contract.
 */
TQ_API tq_status tq_nvfp4_quantize(const void *w, tq_dtype wt, int64_t n, int64_t k, int64_t ldw, uint8_t *codes,
                                   uint8_t *scales, float *tensor_scale, void *stream);

/* tq_nvfp4_dequantize -- w~ in fp32, rounded to ot; the operand rules of
 * tq_dequantize plus the tensor block written by tq_nvfp4_quantize. */
TQ_API tq_status tq_nvfp4_dequantize(const uint8_t *codes, const uint8_t *scales, const float *tensor_scale,
                                     int64_t n, int64_t k, void *w_out, tq_dtype ot, int64_t ldo, void *stream);

/*
 * tq_nvfp4_gemm -- Y[i][r] = sum_k w~[r][k] X[i][k] for i < m <= 32 with the
 * fused kernel of tq_gemm: codes enter the tensor cores as fp16 E2M1 values,
 * the activation as fp16 (converted once per call, no rotation), each
 * 16-column partial sum is scaled by its E4M3 block scale in fp32 and the
 * row total by g.  Workspace: tq_gemm_workspace_bytes(m, n, k), same rules.
 * m > 32 returns TQ_ERR_SHAPE.
 */
TQ_API tq_status tq_nvfp4_gemm(const uint8_t *codes, const uint8_t *scales, const float *tensor_scale, int64_t n,
                               int64_t k, const void *X, tq_dtype xt, int64_t m, int64_t ldx, void *Y, tq_dtype yt,
                               int64_t ldy, void *workspace, size_t ws_bytes, void *stream);

/* Several NVFP4 products in one launch pair, as tq_gemm_batch. */
typedef struct {
    const uint8_t *codes;
    const uint8_t *scales;
    const float *tensor_scale; /* device tensor block of this matrix */
    int64_t n;
    int64_t k;
    const void *X;
    int64_t ldx;
    void *Y;
    int64_t ldy;
} tq_nvfp4_gemm_desc;

TQ_API size_t tq_nvfp4_gemm_batch_workspace_bytes(const tq_nvfp4_gemm_desc *descs, int count, int64_t m);
TQ_API tq_status tq_nvfp4_gemm_batch(const tq_nvfp4_gemm_desc *descs, int count, int64_t m, tq_dtype xt, tq_dtype yt,
                                     void *workspace, size_t ws_bytes, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Key/value cache in TQ4_1S, and what works on it
 * ---------------------------------------------------------------------------
 * The attention half of a decoding step next to the products above: rotary
 * positions, writing keys and values into a paged cache in the codec of the
 * weights (TQ page, 格式原理), reading them back, attention over the packed
 * records, and moving an accepted branch of drafted tokens together.
 *
 * The cache is a pool of pages that the caller allocates:
 *  - codes   uint8  [pages][2][kv_heads][page_size][head_dim / 2]
 *  - scales  uint16 [pages][2][kv_heads][page_size][head_dim / 16]
 *    plane 0 the keys, plane 1 the values; 5.0 bits per element.
 *  - A record is one token's head vector: per 32-element block of the head
 *    (element index = column index of the sign hash) the codes and scales of
 *    tq_quantize, bit for bit, except that a scale saturates at 23968 (so that
 *    every centroid times its scale is finite in fp16; a block that holds a
 *    NaN gets that scale and code 0).  Byte i of a record's codes holds
 *    elements 2i (low nibble) and 2i + 1; its scales are d0, d1 of each block.
 *  - page_table[b][i] is the page of tokens i * page_size .. of sequence b.  A
 *    token whose column is past pages_per_seq, or whose page id is outside
 *    [0, pages), has no place: writes of it are dropped, reads give zeros, and
 *    attention leaves it out.
 *    Sequences may share pages that are only read; a page that tq_kv_append or
 *    tq_kv_commit writes stands once in the table.
 *  - Sizes: head_dim a multiple of 32 up to TQ_KV_MAX_HEAD_DIM; page_size a
 *    power of two from 16 to TQ_KV_MAX_PAGE; a sequence's table spans at most
 *    2^30 tokens, the whole table TQ_KV_MAX_CAPACITY.  Offsets into the pool
 *    are 64-bit.
 *
 * Head operands (x, k, v, q, out) are [tokens][heads][dim] with unit element
 * stride and the strides given, in elements.
 */
#define TQ_KV_MAX_HEAD_DIM 256
#define TQ_KV_MAX_PAGE 1024
#define TQ_KV_MAX_HEADS 1024
#define TQ_KV_MAX_BATCH 4096
#define TQ_KV_MAX_TREE 64
#define TQ_KV_MAX_LAYERS 4096
#define TQ_KV_MAX_TOKENS ((int64_t)1 << 24)
#define TQ_ROPE_MAX_DIM 1024
#define TQ_KV_MAX_SCALE 65536.0f
#define TQ_KV_MAX_CAPACITY ((int64_t)1 << 34)

typedef struct {
    uint8_t *codes;            /* device, 16-byte aligned */
    uint16_t *scales;          /* device, 16-byte aligned */
    int64_t pages;             /* pages of the pool */
    const int32_t *page_table; /* device, [batch][page_table_ld] */
    int64_t batch;             /* sequences, <= TQ_KV_MAX_BATCH */
    int64_t pages_per_seq;     /* columns of the table in use */
    int64_t page_table_ld;     /* >= pages_per_seq */
    int32_t kv_heads;
    int32_t head_dim;
    int32_t page_size;
} tq_kv_cache;

/* Bytes of a pool's codes (2 * pages * kv_heads * page_size * head_dim / 2)
 * and scales (a quarter of that); 0 for invalid sizes. */
TQ_API size_t tq_kv_codes_bytes(int64_t pages, int64_t kv_heads, int64_t head_dim, int64_t page_size);
TQ_API size_t tq_kv_scales_bytes(int64_t pages, int64_t kv_heads, int64_t head_dim, int64_t page_size);

/* A rotation by positions: the first rot_dim elements of a head in pairs
 * (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved; the rest pass
 * unchanged. */
typedef struct {
    const float *inv_freq; /* device, rot_dim / 2 angles per position, in radians */
    int32_t rot_dim;       /* even, 2 .. dim */
    int32_t interleaved;
    int32_t inverse;       /* rotate back (by minus the angle): the transpose, i.e. the gradient */
    float scale;           /* multiplies cos and sin (1 unless a long-context scaling asks for more) */
} tq_rope_desc;

/*
 * tq_rope -- for pair (x, y) of frequency f at position p, with a = p f:
 *   out = scale * (x cos a - y sin a, x sin a + y cos a)
 * The angle is formed and reduced in 64 bits, so positions of any size keep
 * their accuracy; the rotation is fp32, rounded once to t.
 *   x, out     device, tokens x heads x dim of dtype t, aligned to t (16-byte
 *              alignment and strides that are multiples of 16 bytes run
 *              fastest); out may be x itself (same strides), and must not
 *              overlap it otherwise
 *   positions  device, one per token (any value, also negative)
 */
TQ_API tq_status tq_rope(const void *x, void *out, tq_dtype t, int64_t tokens, int64_t heads, int64_t dim,
                         int64_t x_token_stride, int64_t x_head_stride, int64_t out_token_stride,
                         int64_t out_head_stride, const int32_t *positions, const tq_rope_desc *rope, void *stream);

/*
 * tq_kv_append -- writes the records of `tokens` tokens: token i goes to place
 * places[i] (0-based) of sequence seqs[i].  Tokens without a place (a negative
 * sequence or place among them) are dropped.  Two tokens with the same place
 * in one call leave that record undefined.
 *   k, v       device, tokens x kv_heads x head_dim of dtype t, 16-byte
 *              aligned, strides multiples of 8 elements
 *   rope       host, or NULL: rotates the keys on their way in (fp32, not
 *              rounded before the codec); inverse must be 0
 *   positions  device, the tokens' rotary positions (a drafted token's is its
 *              depth in the tree, not its place); ignored without rope
 */
TQ_API tq_status tq_kv_append(const tq_kv_cache *cache, const int32_t *seqs, const int32_t *places, int64_t tokens,
                              const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                              int64_t v_token_stride, int64_t v_head_stride, tq_dtype t, const int32_t *positions,
                              const tq_rope_desc *rope, void *stream);

/*
 * tq_kv_read -- the inverse: keys and values of the given tokens,
 * x~ = s .* (H c) / 32 in fp32, rounded once to t; zeros for a token without a
 * place.  k and v as in tq_kv_append (written; they must not overlap).
 */
TQ_API tq_status tq_kv_read(const tq_kv_cache *cache, const int32_t *seqs, const int32_t *places, int64_t tokens,
                            void *k, int64_t k_token_stride, int64_t k_head_stride, void *v, int64_t v_token_stride,
                            int64_t v_head_stride, tq_dtype t, void *stream);

/*
 * tq_kv_attention -- attention of `tree` drafted tokens per sequence (1 for
 * plain decoding) over the cache.  Sequence b holds lens[b] tokens, and its
 * drafted tokens' records stand behind them, token i at place lens[b] + i
 * (tq_kv_append them first).  Query head h reads key/value head
 * h / (heads / kv_heads).  Row (b, i, h) attends to all lens[b] tokens, to
 * drafted token i and to its ancestors:
 *   out = sum_j softmax_j(scale * q . k~_j) v~_j
 *   lens     device, [batch] (negative counts as 0)
 *   parents  device, [batch][parents_ld], parents[b][i] the drafted token that
 *            i continues (an earlier one), or -1 where it continues the
 *            sequence; any other value says that token i is not there: it and
 *            its descendants are not attended to and their output is zero.
 *            NULL: a chain, token i continues i - 1
 *   q        device, batch x tree x heads x head_dim of dtype qt, 16-byte
 *            aligned, strides multiples of 8 elements; a row with an
 *            infinity, a NaN, or |q * scale| of 2^40 or |q| of 2^122 and more
 *            answers NaN (zeros, like any other, where it has no token to
 *            attend to)
 *   out      device, same shape, dtype ot, the same rules (written; must not
 *            overlap q or the cache)
 *   heads    query heads, a multiple of kv_heads
 *   scale    any number within +-TQ_KV_MAX_SCALE
 *   workspace  device, >= tq_kv_attention_workspace_bytes(...) bytes, 256-byte
 *            aligned, exclusively owned by this call until it completes on
 *            `stream`; need not be cleared, keeps nothing between calls
 * The rotated query, centroid times scale and the softmax weights enter the
 * tensor cores as fp16, a query row times the softmax's scale and a power of two
 * that brings it into fp16's range; sums, the running maximum and the softmax's
 * sum are fp32.  Products of a centroid and a scale below 2^-14 (records of
 * values below about 1e-5) are multiples of 2^-24, where tq_kv_read gives them
 * exactly.  A record that no row attends to may hold anything; one that some row
 * attends to holds finite scales (tq_kv_append writes no others).
 * tree <= TQ_KV_MAX_TREE.  Up to 16 rows (tree * heads / kv_heads) of a
 * key/value head, and every head_dim other than 64 and 128, run the mma.sync
 * kernel; more rows the tcgen05 kernel, whose waits are bounded: one that
 * expires (after about a second) is recorded in the workspace's status word,
 * see tq_workspace_status, and the outputs are then incomplete.  Two launches.
 */
TQ_API size_t tq_kv_attention_workspace_bytes(int64_t batch, int64_t tree, int64_t heads, int64_t kv_heads,
                                              int64_t head_dim);
TQ_API tq_status tq_kv_attention(const tq_kv_cache *cache, const int32_t *lens, const int32_t *parents,
                                 int64_t parents_ld, const void *q, tq_dtype qt, int64_t q_batch_stride,
                                 int64_t q_token_stride, int64_t q_head_stride, void *out, tq_dtype ot,
                                 int64_t out_batch_stride, int64_t out_token_stride, int64_t out_head_stride,
                                 int64_t tree, int64_t heads, float scale, void *workspace, size_t ws_bytes,
                                 void *stream);

/*
 * tq_kv_commit -- after drafted tokens were accepted: their records move down
 * to where the sequence continues.  path[b][0..] are the accepted tokens of
 * sequence b in order, indices among its drafted tokens, increasing; the
 * branch ends at `steps` or at the first entry that is not above the one
 * before it (-1 by custom).  Record lens[b] + path[b][i] moves to place
 * lens[b] + i, for keys and values of all heads and of `layers` layers whose
 * pools lie code_layer_stride / scale_layer_stride elements apart (multiples
 * of 16 bytes, a pool or more) and share the page table.  lens itself is the caller's to
 * advance.  Records behind the branch keep what they hold.
 */
TQ_API tq_status tq_kv_commit(const tq_kv_cache *cache, int64_t layers, int64_t code_layer_stride,
                              int64_t scale_layer_stride, const int32_t *lens, const int32_t *path, int64_t path_ld,
                              int64_t steps, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TQ_H_ */
