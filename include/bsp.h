/*
 * bsp.h -- C ABI of libbsp.so: the block-scaled precision linear on B200 (sm_100a).
 *
 * The operation is the quantized linear layer Y = X * W^T (+ bias) of a
 * rectified-flow image transformer in the two storage schemes defined on the
 * "BFL (fp8r / nvfp4)" page (Diffusers quantization doc, format bullets):
 *
 *   nvfp4 (ModelOpt layout): `weight` packed E2M1, two values per byte;
 *          `weight_scale` E4M3, one per block of 16 elements along K;
 *          `weight_scale_2` fp32 global scale; `input_scale` fp32 calibrated
 *          activation scale.
 *   fp8r : `weight` E4M3 with one fp32 `weight_scale` per row; activations are
 *          quantized to E4M3 per row at run time.
 *
 * The same page's "Kernels" table pairs each scheme with a fused path: for nvfp4,
 * an activation quantizer followed by a block-scaled FP4 GEMM; for fp8r, a
 * row-scaled FP8 GEMM.  These entry points are that pair of calls for each scheme.
 *
 * Conventions for every call
 *   - All pointers are DEVICE pointers unless stated otherwise, owned by the caller.
 *     The library makes no allocation and keeps no per-call state: what one call
 *     computes depends only on its arguments.  It does keep a little process-wide
 *     state: per device, a status word written by kernels whose bounded wait ran out
 *     (read and cleared by bsp_last_device_status), cached device properties and
 *     kernel attributes, and nvfp4_linear_noalloc's fixed 128 MiB buffer and its cached
 *     address; process-wide, the wait limit (bsp_set_wait_limit_ms) and the kernel
 *     choices that the bsp_testing_set_* hooks of bsp_testing.h switch.  Every tensor
 *     is contiguous row-major.  All work is enqueued asynchronously on `stream`
 *     (NULL = the legacy default stream) of the CURRENT device; nothing synchronises
 *     the host.
 *   - Tensor pointers must be 16-byte aligned (BSP_ERR_MISALIGNED otherwise).
 *   - Argument errors are detected on the host before any launch and returned as a
 *     negative bsp_status; nothing is enqueued in that case.  A zero-sized problem
 *     (M == 0, or N == 0 for a GEMM) returns BSP_OK and enqueues nothing; its
 *     pointers may then be NULL.
 *   - Launch failures return BSP_ERR_CUDA.  Faults found by the kernels themselves
 *     (a bounded wait that ran out) are recorded in a per-device status word and
 *     reported by bsp_last_device_status().
 *   - Only compute capability 10.0 (B200, sm_100a) is supported
 *     (BSP_ERR_UNSUPPORTED_DEVICE otherwise).  There is no fallback path.
 *
 * Number formats
 *   E2M1: sign, 2 exponent bits (bias 1), 1 mantissa bit; magnitudes
 *         {0, 0.5, 1, 1.5, 2, 3, 4, 6}.  Packed two per byte: element 2j in bits 0-3,
 *         element 2j+1 in bits 4-7.
 *   E4M3: the "fn" variant (bias 7, no infinities, max 448, 0x7F/0xFF are NaN).
 *   bf16 in and out.  Rounding everywhere is to nearest, ties to even; encoders
 *   saturate (E2M1 at +-6, E4M3 at +-448) and keep the sign.
 *
 * Scale-factor layouts for NVFP4 block scales (one E4M3 byte per 16 elements):
 *   BSP_SF_LINEAR: [rows][K/16] row-major.
 *   BSP_SF_MMA   : the tiled layout the tensor cores read.  Rows are grouped in
 *                  tiles of 128 and block-columns in tiles of 4; tile (rt, ct) is
 *                  512 contiguous bytes at offset (rt * ceil(K/64) + ct) * 512, and
 *                  inside it row r, block-column c sits at
 *                  (r % 32) * 16 + ((r / 32) % 4) * 4 + (c % 4).
 *                  Its size is nvfp4_sf_bytes(rows, K, BSP_SF_MMA) (rows padded to
 *                  a multiple of 128); padding bytes are never read for results.
 */
#ifndef BSP_H_
#define BSP_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* bsp_stream_t; /* same handle as cudaStream_t */

typedef enum {
    BSP_OK = 0,
    BSP_ERR_INVALID_ARG = -1,       /* null pointer, bad enum, negative size        */
    BSP_ERR_UNSUPPORTED_SHAPE = -2, /* a size outside the documented constraints    */
    BSP_ERR_MISALIGNED = -3,        /* a tensor pointer not 16-byte aligned         */
    BSP_ERR_UNSUPPORTED_DEVICE = -4,/* current device is not compute capability 10.0 */
    BSP_ERR_CUDA = -5,              /* a CUDA runtime call or launch failed          */
    BSP_ERR_TIMEOUT = -6            /* a kernel's bounded wait ran out (device side) */
} bsp_status;

typedef enum { BSP_SF_LINEAR = 0, BSP_SF_MMA = 1 } bsp_sf_layout;

/*
 * nvfp4_quantize_act -- NVFP4 activation quantizer ("BFL (fp8r / nvfp4)", Kernels
 * table: the activations of an nvfp4 linear are quantized before the FP4 GEMM; the
 * format bullet gives block 16, E4M3 block scales and the fp32 `input_scale`).
 *
 *   x_bf16        [M][K] bf16.
 *   global_scale  device pointer to ONE fp32: the decode-side global scale g
 *                 (`input_scale` for activations, `weight_scale_2` for weights).
 *   codes         out [M][K/2] bytes, packed E2M1.
 *   scales        out E4M3 block scales in `layout` (nvfp4_sf_bytes(M, K, layout)).
 * Per block b of 16 elements along K (every step one IEEE binary32 operation):
 *   s_b = amax_b / (6 g) (0 when 6 g is 0) ; scales[b] = E4M3(s_b) ; d = e4m3(scales[b]) * g ;
 *   d == 0 -> all 16 codes 0 ; else code_i = E2M1(x_i * (1/d)), 1/d clamped to FLT_MAX.
 * Constraints: K % 16 == 0; BSP_SF_MMA also needs K % 64 == 0.
 */
int nvfp4_quantize_act(const void* x_bf16, int64_t M, int64_t K, const float* global_scale,
                       uint8_t* codes, uint8_t* scales, int layout, bsp_stream_t stream);

/*
 * nvfp4_gemm -- block-scaled FP4 GEMM with the dequantisation fused into the
 * epilogue ("BFL (fp8r / nvfp4)", Kernels table: the nvfp4 fused GEMM).
 *
 *   a_codes [M][K/2], a_sf (BSP_SF_MMA, rows = M), a_global (device, 1 fp32 = input_scale)
 *   w_codes [N][K/2], w_sf (BSP_SF_MMA, rows = N), w_global (device, 1 fp32 = weight_scale_2)
 *   bias_bf16  [N] bf16 or NULL.
 *   out_bf16   [M][N] bf16.
 *   Y[m][n] = bf16( acc[m][n] * (a_global * w_global) + bias[n] ),
 *   acc = sum_k e2m1(a)*e4m3(sa) * e2m1(w)*e4m3(sw), accumulated in fp32 on the
 *   tensor cores.
 * Constraints: K % 64 == 0, K >= 64; N % 8 == 0.  Any M >= 0.
 * Launch: with programmatic stream serialisation (also fp8r_gemm and nvfp4_gemm_quant).
 * The kernel reads its inputs and writes its output only after the preceding grid on
 * the stream has completed, so this is safe after any kernel; after the library's own
 * quantizer, which triggers early, the GEMM's prologue overlaps the quantizer's tail.
 */
int nvfp4_gemm(const uint8_t* a_codes, const uint8_t* a_sf, const float* a_global,
               const uint8_t* w_codes, const uint8_t* w_sf, const float* w_global,
               const void* bias_bf16, void* out_bf16, int64_t M, int64_t N, int64_t K,
               bsp_stream_t stream);

/*
 * nvfp4_gemm_quant -- nvfp4_gemm whose output is handed straight to the next nvfp4
 * linear: instead of writing Y in bf16, the epilogue quantizes bf16(Y) exactly as
 * nvfp4_quantize_act would (same block-16 arithmetic, global scale out_global) and
 * writes the codes and MMA-layout scales ("BFL (fp8r / nvfp4)", Kernels table: every
 * nvfp4 linear quantizes its activations; in an MLP the second linear's activations
 * are the first one's output).  Bit-identical to nvfp4_gemm followed by
 * nvfp4_quantize_act(Y, out_global, BSP_SF_MMA), without the bf16 round trip.
 *   out_global  device fp32: the next layer's input_scale.
 *   out_codes   [M][N/2] bytes, packed E2M1 ; out_sf  nvfp4_sf_bytes(M, N, BSP_SF_MMA)
 *               bytes (padding rows of the last 128-row tile are not written).
 * Other arguments as nvfp4_gemm.  Constraints: those of nvfp4_gemm and N % 64 == 0.
 * Always runs the CTA-pair kernel.
 */
int nvfp4_gemm_quant(const uint8_t* a_codes, const uint8_t* a_sf, const float* a_global,
                     const uint8_t* w_codes, const uint8_t* w_sf, const float* w_global,
                     const void* bias_bf16, const float* out_global, uint8_t* out_codes,
                     uint8_t* out_sf, int64_t M, int64_t N, int64_t K, bsp_stream_t stream);

/*
 * nvfp4_linear -- the nvfp4 linear forward in one call ("BFL (fp8r / nvfp4)", Kernels
 * table: the activations are quantized at run time, then the fused FP4 GEMM runs):
 * nvfp4_quantize_act(x, input_scale) into `workspace` (BSP_SF_MMA scales), then
 * nvfp4_gemm against the pre-quantized weights.  The GEMM is launched with
 * programmatic stream serialisation, so its prologue overlaps the end of the
 * quantizer; it reads no input before the quantizer has completed.  Results are
 * bit-identical to the two separate calls.
 *
 *   x_bf16        [M][K] bf16 activations.
 *   input_scale   device pointer to one fp32: the activation global scale g.
 *   w_codes, w_sf, w_scale   the quantized weight: [N][K/2] codes, BSP_SF_MMA scales
 *                 (rows = N), device fp32 weight_scale_2.
 *   bias_bf16     [N] bf16 or NULL.   out_bf16  [M][N] bf16.
 *   workspace     caller-owned device buffer of at least
 *                 nvfp4_linear_workspace_bytes(M, K) bytes, 16-byte aligned.  It receives
 *                 the quantized activations (codes, then scales at a 256-byte boundary;
 *                 after them, at the next 256-byte boundary, 8 KB that
 *                 nvfp4_linear_dynamic uses for per-CTA maxima), is overwritten by every
 *                 call, and must not be in use by another call that can run at the same
 *                 time (another stream).
 * Constraints: K % 64 == 0, K >= 64, N % 8 == 0 (those of the two calls).
 * Errors: BSP_ERR_INVALID_ARG when workspace is NULL or workspace_bytes too small;
 * otherwise as nvfp4_quantize_act and nvfp4_gemm.
 */
int nvfp4_linear(const void* x_bf16, const float* input_scale, const uint8_t* w_codes,
                 const uint8_t* w_sf, const float* w_scale, const void* bias_bf16,
                 void* out_bf16, int64_t M, int64_t N, int64_t K, void* workspace,
                 int64_t workspace_bytes, bsp_stream_t stream);

/*
 * nvfp4_linear_dynamic -- nvfp4_linear with the activation global scale computed from
 * this call's activations instead of a calibrated constant ("BFL (fp8r / nvfp4)",
 * nvfp4 bullet: `input_scale` is an fp32 activation scale; here g = amax(x) / (448*6),
 * the global-scale convention used for the weights, the same value nvfp4_global_scale(x)
 * gives), then the nvfp4_linear path with it.  Two launches precede the GEMM: a pass over
 * x leaving one maximum of |x| per CTA in the workspace, and the quantizer, whose CTAs
 * reduce those maxima to g themselves; CTA 0 writes g to *input_scale_out, which the GEMM
 * then reads.  input_scale_out is a device fp32 the caller owns (4-byte aligned); it holds
 * g when the call's work completes.  Other arguments, workspace rules and errors as
 * nvfp4_linear.  Costs one more read of x than nvfp4_linear.
 */
int nvfp4_linear_dynamic(const void* x_bf16, float* input_scale_out, const uint8_t* w_codes,
                         const uint8_t* w_sf, const float* w_scale, const void* bias_bf16,
                         void* out_bf16, int64_t M, int64_t N, int64_t K, void* workspace,
                         int64_t workspace_bytes, bsp_stream_t stream);

/* Workspace bytes nvfp4_linear / nvfp4_linear_dynamic need for an [M][K] activation
 * (codes, padding to 256 bytes, MMA-layout scales, padding to 256 bytes, 8 KB of per-CTA
 * maxima); negative on bad arguments. */
int64_t nvfp4_linear_workspace_bytes(int64_t M, int64_t K);

/*
 * nvfp4_linear_noalloc -- nvfp4_linear without a caller workspace and without any
 * allocation.  The pages have no counterpart: this is a deployment variant of
 * nvfp4_linear for callers that must not allocate device memory after start-up (a
 * serving loop with a fixed memory plan, C code without an allocator): cudaMalloc /
 * cudaFree can synchronise the device and fail under memory pressure.
 *
 * Arguments and results: those of nvfp4_linear minus workspace / workspace_bytes;
 * results are bit-identical to nvfp4_linear.  The quantized activations go to one
 * buffer of nvfp4_linear_noalloc_max_bytes() bytes (128 MiB) per device, compiled
 * into the library (a file-scope __device__ array).
 * Footprint: the buffer takes 128 MiB of device memory on every device where its
 * module is loaded, until the context is destroyed, even in a process that never
 * calls this function: at context creation under CUDA_MODULE_LOADING=EAGER, or at
 * the first call of this function on the device under lazy loading (the default).
 * Its address is looked up on the first call on each device (which may load the
 * module), so make that first call outside any stream capture; a lookup that fails
 * returns BSP_ERR_CUDA, leaves no pending CUDA error, and is retried by the next call.
 * Nothing in it needs to start at zero (each call writes what it reads).
 * Errors: BSP_ERR_UNSUPPORTED_SHAPE when nvfp4_linear_workspace_bytes(M, K) exceeds
 * the buffer; otherwise as nvfp4_linear.
 * Concurrency: the buffer is shared by all calls on a device, so calls that can run
 * at the same time (different streams, unordered host threads) race on it and
 * corrupt each other's results; calls ordered on one stream are safe.
 */
int nvfp4_linear_noalloc(const void* x_bf16, const float* input_scale, const uint8_t* w_codes,
                         const uint8_t* w_sf, const float* w_scale, const void* bias_bf16,
                         void* out_bf16, int64_t M, int64_t N, int64_t K, bsp_stream_t stream);

/* Size in bytes of nvfp4_linear_noalloc's per-device buffer (the largest workspace it
 * accepts). */
int64_t nvfp4_linear_noalloc_max_bytes(void);

/*
 * fp8r_quantize_rows -- per-row E4M3 quantizer ("BFL (fp8r / nvfp4)", fp8r bullet:
 * activations are quantized to E4M3 per row at run time; weights use one fp32 scale
 * per row).
 *   x_bf16 [M][K] bf16 ; q_e4m3 out [M][K] ; row_scale out [M] fp32.
 *   s_m = amax_m / 448 ; s_m == 0 -> q = 0 ; else q = E4M3(x * (1/s_m)), 1/s_m
 *   clamped to FLT_MAX.
 * Constraints: K % 8 == 0.
 */
int fp8r_quantize_rows(const void* x_bf16, int64_t M, int64_t K, uint8_t* q_e4m3,
                       float* row_scale, bsp_stream_t stream);

/*
 * fp8r_gemm -- row-scaled FP8 GEMM ("BFL (fp8r / nvfp4)", Kernels table: the fp8r
 * fused GEMM with per-row scales).
 *   a_e4m3 [M][K], a_row_scale [M]; w_e4m3 [N][K], w_row_scale [N]; bias [N] or NULL.
 *   Y[m][n] = bf16( (acc[m][n] * sA[m]) * sW[n] + bias[n] ), acc in fp32 on the
 *   tensor cores.
 * Constraints: K % 16 == 0, K >= 16; N % 8 == 0.  Any M >= 0.
 */
int fp8r_gemm(const uint8_t* a_e4m3, const float* a_row_scale, const uint8_t* w_e4m3,
              const float* w_row_scale, const void* bias_bf16, void* out_bf16, int64_t M,
              int64_t N, int64_t K, bsp_stream_t stream);

/*
 * fp8r_linear -- the fp8r linear forward in one call ("BFL (fp8r / nvfp4)", fp8r bullet
 * and Kernels table: activations quantized to E4M3 per row at run time, then the
 * row-scaled FP8 GEMM): fp8r_quantize_rows(x) into `workspace`, then fp8r_gemm (launched
 * as the quantizer's programmatic dependent).  Results are bit-identical to the two calls.
 *   x_bf16 [M][K] bf16 ; w_e4m3 [N][K] ; w_row_scale [N] fp32 ; bias [N] bf16 or NULL ;
 *   out_bf16 [M][N].
 *   workspace  caller-owned device buffer of at least fp8r_linear_workspace_bytes(M, K)
 *              bytes, 16-byte aligned (codes, then the row scales at a 256-byte boundary);
 *              fully rewritten by each call; not shared by calls that can run at the same
 *              time.
 * Constraints: those of fp8r_quantize_rows and fp8r_gemm.  Errors as those two, and
 * BSP_ERR_INVALID_ARG for a missing or too small workspace.
 */
int fp8r_linear(const void* x_bf16, const uint8_t* w_e4m3, const float* w_row_scale,
                const void* bias_bf16, void* out_bf16, int64_t M, int64_t N, int64_t K,
                void* workspace, int64_t workspace_bytes, bsp_stream_t stream);

/* Workspace bytes fp8r_linear needs for an [M][K] activation; negative on bad arguments. */
int64_t fp8r_linear_workspace_bytes(int64_t M, int64_t K);

/*
 * nvfp4_global_scale -- g = amax(X) / (448 * 6) over n bf16 values, written to the
 * device fp32 at `global_scale_out` (the nvfp4 `weight_scale_2` / `input_scale`
 * convention: a decode-side multiplier that maps the largest block scale to the
 * E4M3 maximum).  Enqueues a clear of the output, an atomic max over the input and a
 * final divide; no scratch memory.  Constraints: n % 8 == 0.
 */
int nvfp4_global_scale(const void* x_bf16, int64_t n, float* global_scale_out,
                       bsp_stream_t stream);

/*
 * nvfp4_dequantize -- decode NVFP4 to bf16: the weight decode of the dequantise-only
 * fallback ("BFL (fp8r / nvfp4)", closing paragraph of the "Kernels" section: weights are
 * dequantized back to bf16 and the GEMM runs in bf16 on activations that are not
 * quantized, so results differ slightly from the fused path).  Per element, in binary32
 * with round to nearest even and no flush to zero:
 *     out = bf16_rne( (e2m1(code) * e4m3(scale)) * g )
 * (the first product is exact).  Not on the fused hot path; provided for comparison and
 * for callers that need bf16 weights.
 *   codes         [rows][K/2] packed E2M1 (element 2j in the low nibble)
 *   scales        E4M3 block scales in `layout` (BSP_SF_LINEAR [rows][K/16] or BSP_SF_MMA)
 *   global_scale  device fp32, 1 element (weight_scale_2 or input_scale)
 *   out_bf16      [rows][K] bf16, caller-owned
 * Constraints: K % 16 == 0 (K % 64 == 0 for BSP_SF_MMA); codes and out 16-byte aligned,
 * global_scale 4-byte aligned; scale bytes finite (a NaN scale gives NaN elements).
 * Errors: BSP_ERR_INVALID_ARG, BSP_ERR_UNSUPPORTED_SHAPE, BSP_ERR_MISALIGNED,
 * BSP_ERR_UNSUPPORTED_DEVICE, BSP_ERR_CUDA.  Asynchronous on `stream`; no allocation.
 */
int nvfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int layout,
                     const float* global_scale, int64_t rows, int64_t K, void* out_bf16,
                     bsp_stream_t stream);

/*
 * nvfp4_gemv -- a few rows of bf16 activations against an NVFP4 weight, the activations NOT
 * quantized to it: the product of the dequantise-only path ("BFL (fp8r / nvfp4)", closing paragraph
 * of the "Kernels" section) for single tokens, read straight from the 4-bit weight.
 *   x_bf16  [M][K] bf16, 1 <= M <= 32 (M == 0 returns BSP_OK).
 *   w_codes [N][K/2], w_sf (BSP_SF_MMA, rows = N), w_scale (device, 1 fp32), bias_bf16 [N] or
 *           NULL, out_bf16 [M][N]: as nvfp4_gemm (block scales have no sign).
 *   Y[m][n] = bf16( w_scale * sum_k x[m][k] * e2m1(w[n][k]) * e4m3(sf[n][k/16]) + bias[n] ),
 *   sums in fp32.  x reaches the tensor cores in f16 times a power of two for each row: elements down
 *   to 2^-28 of the row's largest exactly, smaller ones to 2^-39 of it.  A row that holds an infinity or
 *   a NaN gives NaN.  The rows do not affect one another.  out must not overlap x.
 *   workspace  device buffer of at least nvfp4_gemv_workspace_bytes(M, N, K) bytes, 16-byte
 *              aligned, any contents; not shared by calls that can run at the same time.
 * Constraints: K % 64 == 0, K >= 64; N % 8 == 0; M <= 32 (BSP_ERR_UNSUPPORTED_SHAPE).  A large
 * weight takes 1.2 to 1.9 times as long as reading it with up to 8 rows, 1.7 to 2.4 times with 16 and 2.7
 * to 3.8 times with 32.  nvfp4_linear, which quantizes x, is then the faster form: from 16 rows on at
 * 131072 x 8192, from some 26 at 16384 x 12288, at no number of rows up to 4096 x 14336.
 */
int nvfp4_gemv(const void* x_bf16, const uint8_t* w_codes, const uint8_t* w_sf,
               const float* w_scale, const void* bias_bf16, void* out_bf16, int64_t M, int64_t N,
               int64_t K, void* workspace, int64_t workspace_bytes, bsp_stream_t stream);

/* Workspace bytes nvfp4_gemv needs; negative on bad arguments. */
int64_t nvfp4_gemv_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * The block-scaled 8-bit key/value cache.  One cache (one layer) is four device arrays:
 *   k_cache, v_cache  E4M3 codes [pages][Hkv][page_size][D]
 *   k_scale, v_scale  E8M0 bytes [pages][Hkv][page_size / 16]: one power of two 2^(byte - 127)
 *                     for each block of 16 tokens and head; value = code * scale.
 * and the ragged batch of a step is described, for both calls, by
 *   block_table [B][max_pages] int32: token t of sequence b lies in page
 *               block_table[b][t / page_size], slot t % page_size;
 *   cu_new      [B + 1] int32, ascending from 0: the new tokens of sequence b are rows
 *               cu_new[b] .. cu_new[b + 1) of q, k, v and out (none, one or many); rows from
 *               cu_new[B] to T are neither read nor written;
 *   kv_len      [B] int32: the sequence's length INCLUDING its new tokens, whose positions are
 *               kv_len[b] - n .. kv_len[b] - 1.
 * Lengths, rows and pages are read on the device, so a captured graph can be replayed while
 * they change.  The kernels keep every access inside the arrays whatever these hold: rows
 * outside [0, T) are cut off; of a sequence whose length is outside [0, max_pages * page_size]
 * fp8kv_append stores nothing and fp8kv_attention reads what the table holds; a page outside
 * [0, pages) is not touched (its tokens are neither stored nor attended to).  Such lengths and pages
 * are reported by bsp_last_device_status() as BSP_ERR_INVALID_ARG.  Table entries of pages that a
 * call does not reach are not read, and of a sequence without new tokens neither the length nor the
 * table is looked at.
 * Constraints: D % 16 == 0, D <= 256; page_size % 16 == 0, page_size <= 4096; Hq % Hkv == 0,
 * Hq and Hkv <= 4096; B <= 2^20, T <= 2^24, T * Hq <= 2^30; max_pages * page_size <= 2^30.
 */

/*
 * fp8kv_append -- rotary positions on the new tokens' q and k, then k and v into the cache, in
 * one launch.
 *   q_bf16   [T][Hq][D] or NULL (nothing is rotated into q_out then), k_bf16, v_bf16 [T][Hkv][D];
 *            *_stride: elements between tokens (% 8 == 0, at least heads * D), so that the three
 *            may lie in one projection's output.
 *   inv_freq [rot / 2] fp32 (device), rot % 16 == 0, 0 <= rot <= D: the first rot elements of each
 *            head are rotated by theta = position * inv_freq[j], taken in 64 bits and reduced there to
 *            an fp32 number of half turns (off by 10^-7 radians at most); any scaling for
 *            long contexts is in the frequencies.  Pairs are (j, j + rot / 2), or (2j, 2j + 1) with
 *            interleaved = 1.  cos and sin are multiplied by rope_scale.
 *   q_out    [T][Hq][D] bf16, contiguous; may be q itself when that is contiguous.
 * For each block of 16 tokens and head (x: the rotated keys in fp32, or the values):
 *   e = ceil(log2(amax / 448)) + 127 over the new tokens, within [0, 246] (0 when amax is 0); a
 *   block that already holds tokens keeps the larger of e and its own (255, a NaN, too), and codes that it holds
 *   move to a raised scale by one rounding; code = E4M3(x * 2^(127 - e)), to nearest even,
 *   saturating at +-448.  Infinities store as +-448 * 2^119, a NaN stores as NaN (only its own
 *   element).
 * Tokens of the block after the last new one are left as they are.  A page that is appended to
 * must belong to one sequence of the batch; a sequence with kv_len[b] < n is left out and reported
 * (neither stored nor, in q_out, rotated).
 */
int fp8kv_append(const void* q_bf16, int64_t q_stride, const void* k_bf16, int64_t k_stride,
                 const void* v_bf16, int64_t v_stride, const float* inv_freq, int64_t rot,
                 int interleaved, float rope_scale, void* q_out_bf16, uint8_t* k_cache,
                 uint8_t* v_cache, uint8_t* k_scale, uint8_t* v_scale, int64_t pages,
                 int64_t page_size, const int32_t* block_table, int64_t max_pages,
                 const int32_t* cu_new, const int32_t* kv_len, int64_t B, int64_t T, int64_t Hq,
                 int64_t Hkv, int64_t D, bsp_stream_t stream);

/*
 * fp8kv_attention -- attention of the new tokens over the cache (which already holds them):
 *   out[r][h] = sum_t p_t v_t / sum_t p_t, p_t = exp(sm_scale * q[r][h] . k_t), head h reading key
 *   head h / (Hq / Hkv), over the tokens t <= pos(r), and t > pos(r) - window when window > 0.
 *   q_bf16  [T][Hq][D], q_stride elements between tokens (% 8 == 0).
 *   out     [T][Hq][D] bf16, contiguous; lse [T][Hq] fp32 or NULL: log of sum_t p_t.
 *   A row that sees no token gives zeros and lse = -infinity.  Softmax statistics and sums are
 *   fp32; q is held to 2^-25 of the largest element of its head (bf16 elements above 2^-17 of that
 *   exactly), and a weight p times the scale of its block of values is rounded once, to 11 bits, or to
 *   2^-32 of the row's largest such product where it is below 2^-21 of that.  All scale bytes are
 *   read as 2^(byte - 127), 255 as NaN.  What masked tokens hold (NaN, stale bytes, stale scales of blocks
 *   behind the end) has no effect.  out must not overlap q or the cache.
 *   workspace  device buffer of at least fp8kv_attention_workspace_bytes(T, Hq, Hkv, D) bytes,
 *              16-byte aligned, any contents; not shared by calls that can run at the same time.
 * Meant for one to a few new tokens per sequence: every 8 or 16 rows (new tokens * Hq / Hkv) of a
 * sequence read its keys and values once more.  Constraint besides the cache's: pages * Hkv < 2^31.
 */
int fp8kv_attention(const void* q_bf16, int64_t q_stride, const uint8_t* k_cache,
                    const uint8_t* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                    int64_t pages, int64_t page_size, const int32_t* block_table,
                    int64_t max_pages, const int32_t* cu_new, const int32_t* kv_len, int64_t B,
                    int64_t T, int64_t Hq, int64_t Hkv, int64_t D, float sm_scale,
                    int64_t window, void* out_bf16, float* lse, void* workspace,
                    int64_t workspace_bytes, bsp_stream_t stream);

/* Workspace bytes fp8kv_attention needs; negative on bad arguments. */
int64_t fp8kv_attention_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D);

/*
 * nvfp4_sf_convert -- re-lay block scales between BSP_SF_LINEAR and BSP_SF_MMA
 * (rows x K/16 bytes; padding of an MMA-layout destination is written as 0).
 * Constraints: K % 64 == 0.  src and dst must not overlap.
 */
int nvfp4_sf_convert(const uint8_t* src, uint8_t* dst, int64_t rows, int64_t K, int from,
                     int to, bsp_stream_t stream);

/* Bytes of a scale array of `rows` x K/16 in `layout`; negative on bad arguments. */
int64_t nvfp4_sf_bytes(int64_t rows, int64_t K, int layout);

/*
 * bsp_last_device_status -- synchronises `stream`, returns and clears the status
 * word the kernels of the current device write (BSP_OK, or BSP_ERR_TIMEOUT when a
 * bounded wait inside a GEMM ran out).  BSP_ERR_CUDA if the synchronisation fails.
 */
int bsp_last_device_status(bsp_stream_t stream);

/* Bounded-wait limit of the GEMM kernels in milliseconds (default 2000, also set by
 * the BSP_WAIT_LIMIT_MS environment variable at first use): the longest any one wait on a
 * pipeline stage or tile may take.  (The fp8r kernel's last-tile helpers wait once for the
 * whole GEMM's issue; that wait is bounded by the larger of this limit and 60 s.)  Returns
 * the old value. */
int64_t bsp_set_wait_limit_ms(int64_t ms);

/* Human-readable name of a bsp_status value. */
const char* bsp_status_string(int status);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int bsp_version(void);

#ifdef __cplusplus
}
#endif

#endif /* BSP_H_ */
