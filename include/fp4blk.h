/*
 * fp4blk.h -- C ABI of libfp4blk: block-scaled 4-bit (NVFP4, MXFP4)
 * quantization and the quantized linear-layer GEMMs it feeds, for AMD
 * Instinct MI355X (gfx950).
 *
 * Formats (pages cited by title and section):
 *  - NVFP4: "NVFP4" (newton.com.tw wiki), section "Technical principle".
 *    E2M1 elements (1 sign, 2 exponent, 1 mantissa bit; values
 *    {0, 0.5, 1, 1.5, 2, 3, 4, 6} and their negatives), 16-element micro-blocks
 *    each with one E4M3 (OCP E4M3FN: bias 7, largest 448, no infinities) scale
 *    byte, and one FP32 scale per tensor: 4.5 bits per value.
 *  - MXFP4: edge-FP4 article (eefocus.com), section "FP4 as the next core
 *    standard".  OCP MX block floating point: 32-element blocks, one E8M0 byte
 *    (2^(byte-127)) per block, E2M1 elements: 4.25 bits per value.
 *  - W4A16 / W4A4: Unsloth Dynamic NVFP4 article (aixq.cc), section "Core
 *    difference: W4A4 vs W4A16".  W4A16 multiplies 4-bit weights, widened to
 *    16 bits, by 16-bit activations; W4A4 quantizes the activations to 4 bits
 *    as well.
 *
 * Packed layout (every packed tensor, row-major, blocks along the last axis):
 *  - codes  uint8 [rows][cols/2]: element (r, c) is in byte r*cols/2 + c/2, in
 *           the low nibble when c is even and the high nibble when c is odd;
 *           nibble = sign<<3 | magnitude index into the grid above.
 *  - scales uint8 [rows][cols/16] (NVFP4, E4M3FN bytes) or [rows][cols/32]
 *           (MXFP4, E8M0 bytes).
 *  - tscale float32 [1] (per tensor) or [rows] (per row): the NVFP4 second-level
 *           scale; value = E2M1(code) * E4M3(scale byte) * tscale.
 * A GEMM computes C[m][n] = sum_k A[m][k] * W[n][k] (C = A . W^T) with W [N][K]
 * packed as above and blocks running along K.
 *
 * Quantization recipe (NVFP4):
 *   tscale    = fl32(amax / 2688)                      (2688 = 6 * 448)
 *   scale[b]  = E4M3 round-to-nearest-even, saturating at 448, of
 *               fl32(block_amax / fl32(6 * tscale)); 0x00 for an all-zero block
 *   code      = E2M1 round-to-nearest-even (ties to the even mantissa bit),
 *               saturating at 6, of fl32(x / fl32(E4M3(scale[b]) * tscale));
 *               a signed zero when that divisor is zero
 * MXFP4: k = floor(log2 block_amax) - 2 (FP4_MX_OCP_FLOOR) or the smallest k
 * with 6 * 2^k >= block_amax (FP4_MX_CEIL), clamped to [-127, 127]; scale byte
 * k + 127 (0 for an all-zero block); code = E2M1-RNE-saturating(x * 2^-k).
 *
 * Conventions:
 *  - Every data pointer is a DEVICE pointer owned by the caller.  The library
 *    allocates and frees nothing.  Its only global state is per-device and
 *    written once per device with atomics (whether the device is a gfx950, its
 *    CU count, which kernels had their LDS limit raised, the device address of
 *    the scratch array of gemm_w4a4_noalloc), plus that scratch array itself;
 *    calls are thread-safe, except that calls of gemm_w4a4_noalloc that
 *    overlap on one device share its scratch.
 *  - Every call is asynchronous on `stream` (0 = the null stream) and never
 *    synchronizes the host.
 *  - Arguments are validated on the host before anything is launched; on an
 *    error nothing is launched and the outputs are untouched.  Validation:
 *    non-null pointers, all sizes > 0, leading dimensions >= the row length,
 *    cols (or K) a multiple of 16 (NVFP4) / 32 (MXFP4), 16-byte aligned base
 *    pointers and leading dimensions that keep every row 16-byte aligned,
 *    workspace at least the queried size.
 *  - Launch failures return FP4_ERR_HIP.  Non-finite inputs (NaN, Inf) violate
 *    a precondition: outputs are unspecified and, if `nonfinite` is non-null,
 *    the device int it points to is set to 1 (it is never cleared by the
 *    library).
 *  - No C++ exception crosses this interface.
 */
#ifndef FP4BLK_H
#define FP4BLK_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FP4_OK = 0,
    FP4_ERR_NULL = 1,               /* a required pointer is null */
    FP4_ERR_SHAPE = 2,              /* a size is <= 0, or not a whole number of blocks */
    FP4_ERR_LAYOUT = 3,             /* leading dimension too small, or misaligned pointer/row */
    FP4_ERR_DTYPE = 4,              /* unknown dtype / mode / rule value */
    FP4_ERR_WORKSPACE = 5,          /* workspace null or smaller than the queried size */
    FP4_ERR_NO_DEVICE = 6,          /* no HIP device is visible */
    FP4_ERR_UNSUPPORTED_DEVICE = 7, /* the current device is not gfx950 */
    FP4_ERR_HIP = 8                 /* a HIP call or kernel launch failed */
} fp4_status;

typedef enum { FP4_F32 = 0, FP4_BF16 = 1 } fp4_dtype;
typedef enum { FP4_SCALE_PER_TENSOR = 0, FP4_SCALE_PER_ROW = 1 } fp4_scale_mode;
typedef enum { FP4_MX_OCP_FLOOR = 0, FP4_MX_CEIL = 1 } fp4_mx_rule;

/* Human-readable name of a status code (static string; never null). */
const char *fp4_status_str(int status);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int fp4blk_version(void);

/* FP4_OK if the current HIP device is a gfx950, else NO_DEVICE / UNSUPPORTED_DEVICE. */
fp4_status fp4blk_check_device(void);

/* ------------------------------------------------------------ NVFP4 ------ */

/* Workspace bytes nvfp4_quantize needs (0 for FP4_SCALE_PER_ROW). */
size_t nvfp4_quantize_workspace(int64_t rows, int64_t cols, fp4_scale_mode mode);

/* NVFP4 quantize ("NVFP4", Technical principle: two-level micro-block scaling).
 *  x        [rows][ldx] fp32 or bf16 (xt), cols % 16 == 0, read only.
 *  codes    [rows][cols/2] out; scales [rows][cols/16] out (E4M3FN bytes).
 *  tscale   out: [1] for FP4_SCALE_PER_TENSOR (amax over the whole tensor),
 *           [rows] for FP4_SCALE_PER_ROW (each row is its own tensor).
 *  ws       device scratch of nvfp4_quantize_workspace() bytes (per-tensor mode).
 *  nonfinite optional device int32 flag, set to 1 if x holds NaN/Inf.
 * Codes and scale bytes equal the recipe above bit for bit. */
fp4_status nvfp4_quantize(const void *x, fp4_dtype xt, int64_t rows, int64_t cols, int64_t ldx,
                          uint8_t *codes, uint8_t *scales, float *tscale, fp4_scale_mode mode,
                          void *ws, size_t ws_bytes, int32_t *nonfinite, hipStream_t stream);

/* NVFP4 dequantize ("NVFP4", Technical principle: a value is its E2M1 element
 * times its micro-block's E4M3 scale times the FP32 tensor scale; the W4A16
 * path of the aixq.cc article, "Core difference: W4A4 vs W4A16", restores the
 * weights to 16 bits this way):
 *  y = fl32(fl32(E2M1(c) * E4M3(s)) * tscale) (the inner product is exact),
 *  stored as fp32 or rounded to nearest even into bf16 (yt).
 *  codes [rows][cols/2], scales [rows][cols/16], tscale [1] (FP4_SCALE_PER_TENSOR)
 *  or [rows] (FP4_SCALE_PER_ROW): device, read only.  cols % 16 == 0.
 *  y [rows][ldy] out (ldy >= cols, 16-byte aligned rows), caller-owned.
 * Errors (host, nothing launched): FP4_ERR_NULL, FP4_ERR_SHAPE, FP4_ERR_LAYOUT,
 * FP4_ERR_DTYPE as for nvfp4_quantize. */
fp4_status nvfp4_dequantize(const uint8_t *codes, const uint8_t *scales, const float *tscale,
                            fp4_scale_mode mode, int64_t rows, int64_t cols, void *y,
                            fp4_dtype yt, int64_t ldy, hipStream_t stream);

/* W4A16 GEMM (aixq.cc article, "Core difference: W4A4 vs W4A16"): C = A . W^T.
 *  a        [M][lda] bf16 activations.
 *  w_*      W [N][K] NVFP4 with a per-tensor scale (w_tscale[1]).
 *  c        [M][ldc] out, fp32 or bf16 (ct; bf16 by round to nearest even).
 * Each weight is widened exactly to E2M1 * E4M3 in bfloat16, products are
 * accumulated in fp32 and the sum is multiplied by w_tscale.  |C - C_exact|
 * stays within 2e-3 * sum_k |a w| (C_exact: fp64 over the dequantized W). */
fp4_status gemm_w4a16(const void *a, int64_t M, int64_t K, int64_t lda, const uint8_t *w_codes,
                      const uint8_t *w_scales, const float *w_tscale, int64_t N, void *c,
                      fp4_dtype ct, int64_t ldc, hipStream_t stream);

/* Decode layout of an NVFP4 weight (for gemm_w4a16_decode).  K is cut into
 * 128-element segments; the layout stores them segment-major,
 *   codes_p  uint8 [K/128][N][64]: byte (s*N + n)*64 + b = codes[n][64*s + b]
 *   scales_p uint8 [K/128][N][8]:  byte (s*N + n)*8 + b  = scales[n][8*s + b]
 * so the 16 rows of a matrix-core tile at one segment are 1 KiB of
 * consecutive bytes.  Same bytes and byte count as the row-major form (4.5 bits
 * a value); only the order differs.  The tensor scale is unchanged.
 * nvfp4_pack_decode rewrites row-major codes [N][K/2] / scales [N][K/16] into
 * it (K % 128 == 0; outputs of N*K/2 and N*K/16 bytes, not overlapping the
 * inputs). */
fp4_status nvfp4_pack_decode(const uint8_t *codes, const uint8_t *scales, int64_t N, int64_t K,
                             uint8_t *codes_p, uint8_t *scales_p, hipStream_t stream);

/* W4A16 (aixq.cc article, "Core difference: W4A4 vs W4A16") on a weight in the
 * decode layout: C = A . W^T, K % 128 == 0.  1 <= M <= 16 (any such K) runs the
 * decode GEMV; larger M the prefill GEMM reading the same layout (the result
 * gemm_w4a16 gives on the row-major weight, bit for bit), so one packed weight
 * serves both.  Same arithmetic and tolerance as gemm_w4a16 (each weight widened
 * exactly to E2M1 * E4M3 in bfloat16, fp32 accumulation, times w_tscale).
 * FP4_ERR_SHAPE, checked on the host before anything is launched, for any M
 * when A spans 2 GiB or more (M * lda * 2 or (M - 1) * lda * 2 + 2 K bytes) or
 * the weight codes do (N * K / 2 bytes): both kernels address the operands with
 * 32-bit byte offsets. */
fp4_status gemm_w4a16_decode(const void *a, int64_t M, int64_t K, int64_t lda, const uint8_t *w_codes_p,
                             const uint8_t *w_scales_p, const float *w_tscale, int64_t N, void *c,
                             fp4_dtype ct, int64_t ldc, hipStream_t stream);

/* Workspace bytes gemm_w4a4 needs: A's codes | scales | tscale, each starting
 * at a 256-byte boundary, in that order (offsets by gemm_w4a4_workspace_offsets). */
size_t gemm_w4a4_workspace(int64_t M, int64_t K, fp4_scale_mode a_mode);
void gemm_w4a4_workspace_offsets(int64_t M, int64_t K, size_t *codes_off, size_t *scales_off,
                                 size_t *tscale_off);

/* W4A4 NVFP4 GEMM (aixq.cc article, "Core difference"): the bf16 activations
 * are quantized to NVFP4 on the device (a_mode: per row, each row its own
 * tensor, or per tensor) into `ws`, then C = A_q . W^T with both operands
 * widened exactly to bfloat16, fp32 accumulation, and the epilogue multiplies
 * by the activation scale (per row) and the weight tensor scale.  After the call
 * `ws` holds A's packed NVFP4 form (codes, scales, tscale) at the documented
 * offsets.  Same tolerance as gemm_w4a16, against fp64 over the two dequantized
 * operands. */
fp4_status gemm_w4a4(const void *a, int64_t M, int64_t K, int64_t lda, fp4_scale_mode a_mode,
                     const uint8_t *w_codes, const uint8_t *w_scales, const float *w_tscale,
                     int64_t N, void *c, fp4_dtype ct, int64_t ldc, void *ws, size_t ws_bytes,
                     hipStream_t stream);

/* The GEMM half of gemm_w4a4 on an already-quantized A (codes [M][K/2],
 * scales [M][K/16], a_tscale [1] or [M] per a_mode). */
fp4_status gemm_nvfp4_w4a4_prequant(const uint8_t *a_codes, const uint8_t *a_scales,
                                    const float *a_tscale, fp4_scale_mode a_mode, int64_t M,
                                    int64_t K, const uint8_t *w_codes, const uint8_t *w_scales,
                                    const float *w_tscale, int64_t N, void *c, fp4_dtype ct,
                                    int64_t ldc, hipStream_t stream);

/* NVFP4 W4A4 with W in the decode layout (nvfp4_pack_decode): the same result as
 * gemm_w4a4 / gemm_nvfp4_w4a4_prequant on the row-major W, bit for bit; each
 * 64-element K stage then reads a weight panel whose rows are 64 bytes apart
 * instead of K/2.  K % 128 == 0, M * K / 2 and N * K / 2 below 2^31
 * (FP4_ERR_SHAPE otherwise, checked before A is quantized); other arguments,
 * workspace and errors as those two. */
fp4_status gemm_w4a4_seg(const void *a, int64_t M, int64_t K, int64_t lda, fp4_scale_mode a_mode,
                         const uint8_t *w_codes_p, const uint8_t *w_scales_p, const float *w_tscale, int64_t N,
                         void *c, fp4_dtype ct, int64_t ldc, void *ws, size_t ws_bytes, hipStream_t stream);

/* For callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): gemm_w4a4 with A's
 * packed NVFP4 form kept in the library's own device scratch instead of a
 * caller's workspace.  The scratch is 32 MiB (33,554,432 bytes) per device, held
 * from the time the library's code is loaded on the device until the process
 * ends.  Arguments as gemm_w4a4 without ws / ws_bytes (W row-major); the result
 * is gemm_w4a4's, bit for bit.  FP4_ERR_WORKSPACE when gemm_w4a4_workspace(M, K,
 * a_mode) exceeds 32 MiB (M * K up to about 29.6 million with per-row scales),
 * checked on the host before anything is launched; other errors as gemm_w4a4.
 * The call allocates and frees nothing.  Every call on a device uses that
 * device's one scratch: calls that overlap on one device (two streams, or two
 * host threads without ordering) race and give unspecified results; calls
 * ordered on one stream do not.  A's packed form stays in the scratch until the
 * next call, but its address is not part of this interface. */
fp4_status gemm_w4a4_noalloc(const void *a, int64_t M, int64_t K, int64_t lda, fp4_scale_mode a_mode,
                             const uint8_t *w_codes, const uint8_t *w_scales, const float *w_tscale, int64_t N,
                             void *c, fp4_dtype ct, int64_t ldc, hipStream_t stream);
fp4_status gemm_nvfp4_w4a4_prequant_seg(const uint8_t *a_codes, const uint8_t *a_scales, const float *a_tscale,
                                        fp4_scale_mode a_mode, int64_t M, int64_t K, const uint8_t *w_codes_p,
                                        const uint8_t *w_scales_p, const float *w_tscale, int64_t N, void *c,
                                        fp4_dtype ct, int64_t ldc, hipStream_t stream);

/* ------------------------------------------------------------ MXFP4 ------ */

/* MXFP4 quantize (eefocus.com article, "FP4 as the next core standard").
 *  x [rows][ldx] fp32 or bf16, cols % 32 == 0; codes [rows][cols/2] out;
 *  scales [rows][cols/32] E8M0 out; rule FP4_MX_OCP_FLOOR or FP4_MX_CEIL. */
fp4_status mxfp4_quantize(const void *x, fp4_dtype xt, int64_t rows, int64_t cols, int64_t ldx,
                          uint8_t *codes, uint8_t *scales, fp4_mx_rule rule, int32_t *nonfinite,
                          hipStream_t stream);

/* MXFP4 dequantize (eefocus.com edge-FP4 article, "FP4 as the next core
 * standard": each 32-element block shares one E8M0 power-of-two scale):
 *  y = E2M1(c) * 2^(s-127) (exact when in range), fp32, or bf16 by round to
 *  nearest even; the scale byte 0xFF (E8M0's NaN) gives NaN for its block.  codes [rows][cols/2], scales [rows][cols/32]: device, read
 *  only; cols % 32 == 0.  y [rows][ldy] out (ldy >= cols, 16-byte aligned rows).
 * Errors (host, nothing launched): FP4_ERR_NULL, FP4_ERR_SHAPE, FP4_ERR_LAYOUT,
 * FP4_ERR_DTYPE. */
fp4_status mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                            int64_t cols, void *y, fp4_dtype yt, int64_t ldy, hipStream_t stream);

/* Workspace bytes mxfp4_gemm_w4a4 needs: A's codes | scales, 256-byte aligned. */
size_t mxfp4_gemm_w4a4_workspace(int64_t M, int64_t K);

/* 1 if mxfp4_gemm_w4a4 leaves A's MXFP4 form in its workspace segment-major
 * (codes [K/128][M][64], E8M0 [K/128][M][4], as mxfp4_gemm_w4a4_seg does): when
 * K % 128 == 0 and A's and W's codes are each under 2 GiB.  0: row-major
 * (codes [M][K/2], E8M0 [M][K/32]).  Either way the bytes are those of
 * mxfp4_quantize(A); only their order differs. */
int mxfp4_gemm_w4a4_a_segment_major(int64_t M, int64_t N, int64_t K);

/* MXFP4 W4A4 GEMM: A (bf16) is quantized to MXFP4 with `rule` into `ws`, then
 * C = A_q . W^T on gfx950's block-scaled FP4 matrix instruction (E8M0 scale per
 * 32 K-elements per row, the MX block), fp32 accumulation.  W [N][K] MXFP4.
 * A's form in `ws` is segment-major where mxfp4_gemm_w4a4_a_segment_major says
 * so (the kernel then reads W's 64-byte row pieces per 128-K segment, A's
 * panels as contiguous runs); the result is the same bit for bit. */
fp4_status mxfp4_gemm_w4a4(const void *a, int64_t M, int64_t K, int64_t lda, fp4_mx_rule rule,
                           const uint8_t *w_codes, const uint8_t *w_scales, int64_t N, void *c,
                           fp4_dtype ct, int64_t ldc, void *ws, size_t ws_bytes,
                           hipStream_t stream);

/* The GEMM half of mxfp4_gemm_w4a4 on an already-quantized A. */
fp4_status mxfp4_gemm_prequant(const uint8_t *a_codes, const uint8_t *a_scales, int64_t M,
                               int64_t K, const uint8_t *w_codes, const uint8_t *w_scales,
                               int64_t N, void *c, fp4_dtype ct, int64_t ldc, hipStream_t stream);

/* MXFP4 W4A16 GEMM (eefocus.com edge-FP4 article, "FP4 as the next core
 * standard": MXFP4 blocks of 32 elements with an E8M0 power-of-two scale; aixq.cc
 * article, "Core difference: W4A4 vs W4A16": 16-bit activations): C = A . W^T
 * with A bf16 [M][lda] and W MXFP4 row-major, codes [N][K/2], E8M0 scales
 * [N][K/32].  Each weight is widened exactly to bf16 (E2M1 times a power of two),
 * fp32 accumulation; no tensor scale.  K % 128 == 0 (FP4_ERR_SHAPE otherwise, and
 * for operands past 2 GiB).  Tolerance as gemm_w4a16. */
fp4_status mxfp4_gemm_w4a16(const void *a, int64_t M, int64_t K, int64_t lda, const uint8_t *w_codes,
                            const uint8_t *w_scales, int64_t N, void *c, fp4_dtype ct, int64_t ldc,
                            hipStream_t stream);

/* Decode layout of an MXFP4 weight: codes as for nvfp4_pack_decode,
 *   codes_p  uint8 [K/128][N][64]: byte (s*N + n)*64 + b = codes[n][64*s + b]
 *   scales_p uint8 [K/128][N][4]:  byte (s*N + n)*4 + b  = scales[n][4*s + b]
 * (the 4 E8M0 bytes of segment s).  Same bytes and count as the row-major form
 * (4.25 bits a value).  K % 128 == 0; outputs of N*K/2 and N*K/32 bytes, not
 * overlapping the inputs. */
fp4_status mxfp4_pack_decode(const uint8_t *codes, const uint8_t *scales, int64_t N, int64_t K,
                             uint8_t *codes_p, uint8_t *scales_p, hipStream_t stream);

/* MXFP4 W4A16 on a weight in the MXFP4 decode layout: C = A . W^T, K % 128 == 0;
 * the decode GEMV for 1 <= M <= 16 (any such K), the prefill GEMM on the same
 * layout for larger M (mxfp4_gemm_w4a16's result, bit for bit).  Arithmetic and
 * tolerance as mxfp4_gemm_w4a16.  FP4_ERR_SHAPE for the same 2 GiB limits as
 * gemm_w4a16_decode, for any M, checked before anything is launched. */
fp4_status mxfp4_gemm_w4a16_decode(const void *a, int64_t M, int64_t K, int64_t lda, const uint8_t *w_codes_p,
                                   const uint8_t *w_scales_p, int64_t N, void *c, fp4_dtype ct, int64_t ldc,
                                   hipStream_t stream);

/* MXFP4 W4A4 GEMM on segment-major operands (eefocus.com edge-FP4 article, "FP4
 * as the next core standard": MXFP4, 32-element blocks with an E8M0 scale).  The
 * same product as mxfp4_gemm_w4a4, bit for bit, with W in the MXFP4 decode layout
 * (mxfp4_pack_decode) instead of row-major: a 256-row panel's 128-element K
 * segment is then contiguous, which is how the kernel reads it.  A (bf16
 * [M][lda]) is quantized with `rule` into `ws` in the same layout (codes
 * [K/128][M][64] at ws, E8M0 [K/128][M][4] at the next 256-byte boundary).
 * K % 128 == 0, M * K / 2 and N * K / 2 below 2^31 (FP4_ERR_SHAPE otherwise,
 * checked before A is quantized); FP4_ERR_WORKSPACE for a null, unaligned or short ws.  C [M][ldc] fp32 or bf16
 * is written; nothing is allocated. */
size_t mxfp4_gemm_w4a4_seg_workspace(int64_t M, int64_t K);
fp4_status mxfp4_gemm_w4a4_seg(const void *a, int64_t M, int64_t K, int64_t lda, fp4_mx_rule rule,
                               const uint8_t *w_codes_p, const uint8_t *w_scales_p, int64_t N, void *c,
                               fp4_dtype ct, int64_t ldc, void *ws, size_t ws_bytes, hipStream_t stream);

/* The GEMM half of mxfp4_gemm_w4a4_seg: A and W both MXFP4 in the segment-major
 * (decode) layout, codes [K/128][rows][64], scales [K/128][rows][4]. */
fp4_status mxfp4_gemm_prequant_seg(const uint8_t *a_codes_p, const uint8_t *a_scales_p, int64_t M, int64_t K,
                                   const uint8_t *w_codes_p, const uint8_t *w_scales_p, int64_t N, void *c,
                                   fp4_dtype ct, int64_t ldc, hipStream_t stream);

/* ---- W4A8: FP4 weights x FP8 activations (eefocus.com edge-FP4 article: an NPU
 * with native W4A8, weights quantized to FP4 and activations to FP8).  Both
 * operands take the OCP MX form: MXFP4 weights, MXFP8 activations. ---- */

/* MXFP8 quantize: x [rows][ldx] (fp32 or bf16) -> codes uint8 [rows][cols]
 * (E4M3FN, sign kept), scales uint8 [rows][cols/32] (E8M0).  Per 32-element
 * block: rule FP4_MX_OCP_FLOOR: 2^k with k = floor(log2 amax) - 8 (the block
 * maximum may saturate at 448); FP4_MX_CEIL: the smallest 2^k with 448 2^k >=
 * amax.  Elements: E4M3 round-to-nearest-even with saturation of |x| / 2^k; a
 * zero block gets scale byte 0.  cols % 32 == 0. */
fp4_status mxfp8_quantize(const void *x, fp4_dtype xt, int64_t rows, int64_t cols, int64_t ldx,
                          uint8_t *codes, uint8_t *scales, fp4_mx_rule rule, int32_t *nonfinite,
                          hipStream_t stream);

/* Workspace bytes mxfp4_gemm_w4a8 needs: A's MXFP8 codes | scales, each at a
 * 256-byte boundary. */
size_t mxfp4_gemm_w4a8_workspace(int64_t M, int64_t K);

/* W4A8 GEMM: the bf16 A is quantized to MXFP8 with `rule` into `ws`, then
 * C = A_q . W^T on gfx950's block-scaled matrix instruction with FP8 and FP4
 * operands (exact products, fp32 accumulation).  W MXFP4 [N][K].  K % 128 == 0,
 * M * K (A's MXFP8 bytes) and N * K / 2 below 2^31 (FP4_ERR_SHAPE otherwise,
 * checked before anything is launched).  Tolerance as the other GEMMs, against
 * fp64 over the dequantized operands. */
fp4_status mxfp4_gemm_w4a8(const void *a, int64_t M, int64_t K, int64_t lda, fp4_mx_rule rule,
                           const uint8_t *w_codes, const uint8_t *w_scales, int64_t N, void *c,
                           fp4_dtype ct, int64_t ldc, void *ws, size_t ws_bytes, hipStream_t stream);

/* The GEMM half of mxfp4_gemm_w4a8 on an already-quantized MXFP8 A (codes
 * [M][K], scales [M][K/32]). */
fp4_status mxfp4_gemm_w4a8_prequant(const uint8_t *a_codes, const uint8_t *a_scales, int64_t M, int64_t K,
                                    const uint8_t *w_codes, const uint8_t *w_scales, int64_t N, void *c,
                                    fp4_dtype ct, int64_t ldc, hipStream_t stream);

/* W4A8 with W in the MXFP4 decode layout (mxfp4_pack_decode: codes [K/128][N][64],
 * scales [K/128][N][4]); A as in mxfp4_gemm_w4a8.  The same result as
 * mxfp4_gemm_w4a8 / _prequant on the row-major W, bit for bit; the weight's
 * 128-element segments are then contiguous panels, which the kernel copies whole.
 * Arguments, workspace and errors as those two. */
fp4_status mxfp4_gemm_w4a8_seg(const void *a, int64_t M, int64_t K, int64_t lda, fp4_mx_rule rule,
                               const uint8_t *w_codes_p, const uint8_t *w_scales_p, int64_t N, void *c,
                               fp4_dtype ct, int64_t ldc, void *ws, size_t ws_bytes, hipStream_t stream);
fp4_status mxfp4_gemm_w4a8_prequant_seg(const uint8_t *a_codes, const uint8_t *a_scales, int64_t M, int64_t K,
                                        const uint8_t *w_codes_p, const uint8_t *w_scales_p, int64_t N, void *c,
                                        fp4_dtype ct, int64_t ldc, hipStream_t stream);

/* ---------------------------------------------------- grouped (MoE) ------ */

/* Grouped GEMMs for mixture-of-experts layers (eefocus.com edge-FP4 article, "FP4
 * as the next core standard": MoE expert weights stored as MXFP4; aixq.cc article
 * on Unsloth's Dynamic NVFP4, throughput section: a mixture-of-experts model run
 * with NVFP4 weights, and all-W4A4 in its "Fast" form).
 *
 * One weight per group (expert), stacked: codes [groups][N][K/2], scales
 * [groups][N][K/16] (NVFP4, E4M3) or [groups][N][K/32] (MXFP4, E8M0), NVFP4
 * tensor scales [groups] floats.  The `rows` grouped rows are the rows of C
 * [rows][ldc]; group e owns rows group_offs[e] .. group_offs[e+1]-1 and
 *   C[t] = A[row_index[t]] . W_e^T      (A[t] when row_index is null),
 * so a router's permutation is applied while A is loaded and C comes out in
 * grouped order.  A has a_rows rows; without row_index a_rows >= rows.
 *
 * group_offs (device, int32 [groups+1]) must be nondecreasing from 0 to rows,
 * and row_index (device, int32 [rows]) entries must lie in [0, a_rows).  Other
 * values give unspecified C but no access outside the buffers: offsets are
 * clamped to [0, rows], and a row index outside A reads as a zero row.  Empty
 * groups are allowed.  rows == 0 returns FP4_OK once groups, group_offs, K, N
 * and the output dtype check out, touching nothing (A, W, C may be null then).
 * groups <= 65536.
 * Errors (checked on the host, nothing launched): FP4_ERR_SHAPE for K not a
 * multiple of 64 (NVFP4) or 128 (MXFP4), A past 2 GiB (its bf16 rows, or for
 * W4A4 its packed codes), one group's weight codes past 2 GiB, or a tile grid of
 * 2^31 workgroups or more; FP4_ERR_NULL, FP4_ERR_LAYOUT as the other GEMMs.
 * nvfp4_grouped_gemm_w4a4 checks all of these before its quantizer runs.
 * Tolerance as the ungrouped GEMMs, row by row. */

/* NVFP4 weights, bf16 A [a_rows][lda]: each weight widened exactly to bf16,
 * fp32 accumulation, times the group's tensor scale. */
fp4_status nvfp4_grouped_gemm_w4a16(const void *a, int64_t a_rows, int64_t K, int64_t lda,
                                    const int32_t *row_index, const int32_t *group_offs, int64_t groups,
                                    int64_t rows, const uint8_t *w_codes, const uint8_t *w_scales,
                                    const float *w_tscale, int64_t N, void *c, fp4_dtype ct, int64_t ldc,
                                    hipStream_t stream);

/* MXFP4 weights, bf16 A: weights widened exactly (E2M1 times a power of two). */
fp4_status mxfp4_grouped_gemm_w4a16(const void *a, int64_t a_rows, int64_t K, int64_t lda,
                                    const int32_t *row_index, const int32_t *group_offs, int64_t groups,
                                    int64_t rows, const uint8_t *w_codes, const uint8_t *w_scales, int64_t N,
                                    void *c, fp4_dtype ct, int64_t ldc, hipStream_t stream);

/* Workspace bytes of nvfp4_grouped_gemm_w4a4: A's per-row NVFP4 form, laid out
 * as gemm_w4a4's per-row workspace for a_rows x K. */
size_t nvfp4_grouped_gemm_w4a4_workspace(int64_t a_rows, int64_t K);

/* NVFP4 W4A4: every A row (token) is quantized once, per row, into `ws`; the
 * grouped GEMM then reads the packed rows through row_index. */
fp4_status nvfp4_grouped_gemm_w4a4(const void *a, int64_t a_rows, int64_t K, int64_t lda,
                                   const int32_t *row_index, const int32_t *group_offs, int64_t groups,
                                   int64_t rows, const uint8_t *w_codes, const uint8_t *w_scales,
                                   const float *w_tscale, int64_t N, void *c, fp4_dtype ct, int64_t ldc, void *ws,
                                   size_t ws_bytes, hipStream_t stream);

/* The GEMM half of nvfp4_grouped_gemm_w4a4 on a per-row NVFP4 A (codes
 * [a_rows][K/2], scales [a_rows][K/16], a_tscale [a_rows]). */
fp4_status nvfp4_grouped_gemm_w4a4_prequant(const uint8_t *a_codes, const uint8_t *a_scales,
                                            const float *a_tscale, int64_t a_rows, int64_t K,
                                            const int32_t *row_index, const int32_t *group_offs,
                                            int64_t groups, int64_t rows, const uint8_t *w_codes,
                                            const uint8_t *w_scales, const float *w_tscale, int64_t N,
                                            void *c, fp4_dtype ct, int64_t ldc, hipStream_t stream);

/* --------------------------------------- key-value cache and attention ---
 *
 * What surrounds the quantized linear layers when a model is served: a paged cache
 * of keys and values, kept in one of the library's block-scaled formats ("NVFP4",
 * Technical principle; edge-FP4 article, eefocus.com, "FP4 as the next core
 * standard" for the E8M0 formats, and "Compute, memory and precision": the decode
 * phase is bound by the bytes it reads, and in long contexts those are the cache's),
 * the attention of a new token that reads it, and the attention of whole prompts.
 *
 * Cache layout.  A page holds page_size tokens of every key head; a token's slot is
 * page * page_size + offset.  Keys and values alike:
 *  - codes  [pages][kv_heads][page_size][row bytes]: FP4_KV_BF16 rows of head_dim
 *           bf16, FP4_KV_MXFP8 head_dim E4M3FN bytes, FP4_KV_NVFP4 / FP4_KV_MXFP4
 *           head_dim/2 bytes (low nibble even);
 *  - scales [pages][kv_heads][head_dim/block][page_size] bytes: E8M0 per 32 values
 *           (MX formats), E4M3FN per 16 (NVFP4); null for FP4_KV_BF16.  Tokens run
 *           along the last axis, so that the scales of neighbouring tokens are read
 *           together;
 *  - tscale [kv_heads] fp32, NVFP4 only: the second-level scale, given by the caller
 *           (a token cannot change it after others are stored).  Finite and >= 0.
 * Blocks run along head_dim; recipes as nvfp4_quantize (with the given tscale: values
 * past 2688 tscale saturate), mxfp4_quantize and mxfp8_quantize.
 *
 * Limits (FP4_ERR_SHAPE): head_dim 64, 128 or 256; page_size a power of two in
 * [16, 256]; pages * page_size < 2^31.  All base pointers 16-byte aligned, all token and
 * head strides (in elements) keep rows of head_dim 16-byte aligned and are >= 0
 * (0 repeats a row; outputs need strides of at least head_dim); the innermost stride
 * is 1.  Other values are FP4_ERR_LAYOUT. */
typedef enum { FP4_KV_BF16 = 0, FP4_KV_MXFP8 = 1, FP4_KV_NVFP4 = 2, FP4_KV_MXFP4 = 3 } fp4_kv_format;

typedef struct {
    fp4_kv_format format;
    int64_t pages, kv_heads, page_size, head_dim;
    void *k_codes, *v_codes;
    uint8_t *k_scales, *v_scales;     /* null for FP4_KV_BF16 */
    const float *k_tscale, *v_tscale; /* FP4_KV_NVFP4 only */
} fp4_kv_cache;

/* Quantize new tokens' keys and values into the cache.
 *  k, v   [tokens][kv_heads][head_dim] fp32 or bf16 (xt), read only, any token and
 *         head stride (rows of a fused projection's output are taken in place).
 *  slots  device int64 [tokens]; a slot outside [0, pages * page_size) skips its token
 *         (padding).  Slots of one call must differ.
 *  rule   of the MX formats' block exponents.  FP4_KV_BF16 stores bf16 inputs bit for
 *         bit and rounds fp32 ones to nearest even.
 *  nonfinite optional device int32, set to 1 if a token that is stored holds NaN/Inf
 *         (quantized formats; their stored values are then unspecified).
 * tokens == 0 returns FP4_OK once the cache, xt and rule check out. */
fp4_status kv_cache_append(const fp4_kv_cache *cache, const void *k, const void *v, fp4_dtype xt,
                           int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                           int64_t v_token_stride, int64_t v_head_stride, const int64_t *slots,
                           fp4_mx_rule rule, int32_t *nonfinite, hipStream_t stream);

/* Read cached sequences back as packed rows of fp32 or bf16 (yt): row t of k and v
 * [tokens][kv_heads][head_dim] is position t - cu_seqlens[b] of sequence b, where
 * cu_seqlens[b] <= t < cu_seqlens[b+1].
 *  block_table device int32 [seqs][table_stride]: page of positions i * page_size ..,
 *         i < table_width.  Entries past a sequence's last page are not read.
 *  cu_seqlens device int32 [seqs+1], nondecreasing.
 * Values as nvfp4_dequantize / mxfp4_dequantize: exact in fp32, bf16 rounded to nearest
 * even.  A row that no sequence holds, or whose page is outside the table or the cache,
 * is zero.  tokens == 0 returns FP4_OK once the other arguments check out. */
fp4_status kv_cache_read(const fp4_kv_cache *cache, const int32_t *block_table, int64_t seqs,
                         int64_t table_width, int64_t table_stride, const int32_t *cu_seqlens,
                         int64_t tokens, void *k, void *v, fp4_dtype yt, int64_t k_token_stride,
                         int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                         hipStream_t stream);

/* Workspace bytes of attn_decode_paged on the current device: 0 when the block table is
 * so narrow that one launch without partial results serves it (ws may be null then), and
 * on bad sizes. */
size_t attn_decode_paged_workspace(int64_t seqs, int64_t heads, const fp4_kv_cache *cache,
                                   int64_t table_width);

/* Attention of one new token per sequence over the cache (its own key and value
 * already appended):  with keys j in [max(0, len - window), len) (window 0: all),
 *   out[b][h] = sum_j softmax_j(scale * q[b][h] . k_j) v_j
 * over the cache's key head h / (heads / kv_heads).  heads % kv_heads == 0.
 *  q      [seqs][heads][head_dim] bf16, any strides as above.
 *  block_table, table_width, table_stride: as kv_cache_read.
 *  seq_lens device int32 [seqs], keys of each sequence, the new one included; clamped
 *         to [0, table_width * page_size].  Length 0 gives a zero row and lse = -inf.
 *         Page ids are clamped into the cache: a bad id gives wrong values, no access
 *         outside the buffers.
 *  scale  in [0, 1e30] (FP4_ERR_SHAPE otherwise); scores past the fp32 range give
 *         unspecified results.
 *  out    [seqs][heads][head_dim] fp32 or bf16 (ot).
 *  lse    optional fp32 [seqs][heads]: log sum_j exp(scale q.k_j), natural logarithm,
 *         with which results over parts of a context can be joined.
 *  ws     attn_decode_paged_workspace() bytes, 16-byte aligned.
 * Scores, softmax sums and output sums are fp32; the softmax weights are rounded to 16
 * bits (bf16; f16, raised by 2^7, for NVFP4) as operands of the matrix core.  Nothing outside a
 * sequence's range is ever used, whatever it holds.  The same inputs give the same
 * bits.  seqs * kv_heads * (table_width * page_size / 128) < 2^31 (FP4_ERR_SHAPE). */
fp4_status attn_decode_paged(const void *q, int64_t seqs, int64_t heads, int64_t q_seq_stride,
                             int64_t q_head_stride, const fp4_kv_cache *cache, const int32_t *block_table,
                             int64_t table_width, int64_t table_stride, const int32_t *seq_lens, float scale,
                             int64_t window, void *out, fp4_dtype ot, int64_t o_seq_stride,
                             int64_t o_head_stride, float *lse, void *ws, size_t ws_bytes, hipStream_t stream);

/* Workspace bytes of attn_prefill on the current device: for a few rows against a long
 * context, whose keys are split among workgroups; 0 otherwise (ws may be null then). */
size_t attn_prefill_workspace(int64_t q_tokens, int64_t heads, int64_t k_tokens, int64_t kv_heads, int64_t head_dim,
                              int64_t seqs);

/* Attention of whole prompts, packed one behind the other.
 *  q      [q_tokens][heads][head_dim], k, v [k_tokens][kv_heads][head_dim], bf16, any
 *         strides as above (token strides of k and v below 2^24 elements: FP4_ERR_LAYOUT);
 *         heads % kv_heads == 0; head_dim 64, 128 or 256.
 *  cu_q, cu_k device int32 [seqs+1], nondecreasing from 0 to q_tokens / k_tokens:
 *         sequence b has lq = cu_q[b+1] - cu_q[b] queries and lk = cu_k[b+1] - cu_k[b]
 *         keys.  The last query stands at the last key (query i at position
 *         i + lk - lq), so a prompt's next chunk attends to what is cached before it.
 *         Other offsets give unspecified results but no access outside the buffers.
 *  causal 0 or 1: key j is seen when j <= position.  window > 0: and when
 *         j > position - window.
 *  scale, out (fp32 or bf16), lse (fp32 [q_tokens][heads]): as attn_decode_paged.  A
 *         query that sees no key gives a zero row and lse = -inf.
 *  ws     attn_prefill_workspace() bytes, 16-byte aligned.
 * An infinity or NaN in k or v reaches only the queries that see its key (in v: only its
 * column of them).  q_tokens == 0 returns FP4_OK once the other arguments check out;
 * k_tokens == 0 gives zero rows.
 * q_tokens * heads / kv_heads and k_tokens < 2^31 (FP4_ERR_SHAPE). */
fp4_status attn_prefill(const void *q, int64_t q_tokens, int64_t heads, int64_t q_token_stride,
                        int64_t q_head_stride, const void *k, const void *v, int64_t k_tokens,
                        int64_t kv_heads, int64_t head_dim, int64_t k_token_stride, int64_t k_head_stride,
                        int64_t v_token_stride, int64_t v_head_stride, const int32_t *cu_q,
                        const int32_t *cu_k, int64_t seqs, float scale, int causal, int64_t window, void *out,
                        fp4_dtype ot, int64_t o_token_stride, int64_t o_head_stride, float *lse, void *ws,
                        size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------- around the attention ---
 *
 * The other steps of serving a layer over the paged cache, so that a generate loop stays on
 * the device (and can be captured): heads normed and rotated between the projection and the
 * cache, pages dealt to growing sequences and taken back, beam search.  The decode phase is
 * bound by the bytes it reads (edge-FP4 article, eefocus.com, "Compute, memory and
 * precision"); steps of many small launches and host round trips would cost more than that.
 *
 * qk_norm_rope: norm and rotation of every head's row, in one pass.  For a row x of q or k,
 *   y = x (mean_d x^2 + eps)^-1/2 w;   the first `rot` values of y then turn in pairs by
 *   t_i = position * freqs[i]:  (y_a cos t_i - y_b sin t_i, y_b cos t_i + y_a sin t_i)
 * with (a, b) = (i, i + rot/2), or (2i, 2i + 1) when interleaved, i < rot/2.
 *  q, k   [tokens][heads][head_dim], [tokens][kv_heads][head_dim] fp32 or bf16 (xt), any
 *         token and head strides as above; kv_heads 0: no k (k, k_out null).
 *  weights fp32 [head_dim], one head's at `stride` elements from the last one's (0: the
 *         same for every head); 16-byte aligned, strides multiples of 4.  eps > 0 (1e-30 to
 *         1e30); eps == 0: rows are not normed, weights are not read and may be null.
 *  positions device int32 [tokens], any values; freqs device fp64 [rot/2] (radians a
 *         position).  Angles are formed and reduced in 64 bits.  rot == 0: no rotation
 *         (positions and freqs may be null).
 *  q_out, k_out fp32 or bf16 (yt), strides as above; the same memory and strides as q, k (with
 *         xt == yt) is allowed, another overlap is not.
 * fp32 throughout, rounded once to yt; finite rows of any size are normed (squares past fp32 are taken of scaled values).
 * head_dim a multiple of 8 up to 512, rot a multiple of
 * 16 up to head_dim, heads and kv_heads up to 65535, tokens < 2^31 (FP4_ERR_SHAPE).  tokens == 0 returns FP4_OK. */
fp4_status qk_norm_rope(const void *q, const void *k, fp4_dtype xt, int64_t tokens, int64_t heads, int64_t kv_heads,
                        int64_t head_dim, int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride,
                        int64_t k_head_stride, const float *q_weight, const float *k_weight,
                        int64_t q_weight_stride, int64_t k_weight_stride, float eps, const int32_t *positions,
                        const double *freqs, int64_t rot, int interleaved, void *q_out, void *k_out, fp4_dtype yt,
                        int64_t qo_token_stride, int64_t qo_head_stride, int64_t ko_token_stride,
                        int64_t ko_head_stride, hipStream_t stream);

/* The same with the keys and the values written into the cache: what qk_norm_rope followed by
 * kv_cache_append does, but the keys are quantized from fp32 (rounded once), and in one
 * launch.  q and k as qk_norm_rope (kv_heads and head_dim are the cache's); v, slots, rule
 * and nonfinite as kv_cache_append. */
fp4_status qk_norm_rope_append(const fp4_kv_cache *cache, const void *q, const void *k, const void *v, fp4_dtype xt,
                               int64_t tokens, int64_t heads, int64_t q_token_stride, int64_t q_head_stride,
                               int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                               int64_t v_head_stride, const float *q_weight, const float *k_weight,
                               int64_t q_weight_stride, int64_t k_weight_stride, float eps,
                               const int32_t *positions, const double *freqs, int64_t rot, int interleaved,
                               const int64_t *slots, fp4_mx_rule rule, int32_t *nonfinite, void *q_out,
                               fp4_dtype yt, int64_t qo_token_stride, int64_t qo_head_stride, hipStream_t stream);

/* Pages that no sequence holds.
 *  free_list device int32 [pages]: the first state[0] entries are free page ids; pages are
 *         taken from the end.
 *  state  device int32 [2]: the number of free pages, and how many sequences kv_pages_extend
 *         has refused (added up, never cleared by the library).
 * pages, page_size: as fp4_kv_cache.  One pool serves the caches of all layers.  Calls that
 * change a pool or a block table are ordered by the caller, like any calls on one memory. */
typedef struct {
    int32_t *free_list;
    int32_t *state;
    int64_t pages, page_size;
} fp4_kv_pages;

/* Workspace bytes of kv_pages_extend: 0 when one launch serves the sizes (ws may be null). */
size_t kv_pages_extend_workspace(int64_t seqs, int64_t tokens);

/* New tokens for sequences: pages dealt, block table extended, slots and positions listed.
 * Sequence b holds seq_lens[b] tokens in row b of the block table and takes new_lens[b]
 * (negative: 0) more, packed one sequence behind the other.
 *  block_table device int32 [seqs][table_stride]: entries of new pages are written, others
 *         left as they are.
 *  tokens slots and positions written; at least the sum of new_lens (known to the caller,
 *         so that nothing waits for the device).  Those past the sum get slot -1, position 0.
 *  lens_out int32 [seqs], state_out int32 [2]: the lengths and the pool's state after; may be
 *         seq_lens and the pool's state themselves.
 *  slots  int64 [tokens] as kv_cache_append; positions int32 [tokens].
 *  cu_q, cu_k optional int32 [seqs+1]: offsets of the new tokens, and of the whole contexts
 *         (lens_out), as attn_prefill and kv_cache_read take them.
 * Pages are dealt in the order of the sequences and their positions.  A sequence that cannot
 * be served whole (too few free pages are left, the table's row is too narrow, its tokens
 * lie past `tokens`, its length is negative) is refused: its length, its row and the pool stay as
 * they are, its slots are -1 (its positions are those it asked for), and state_out[1] counts it.
 * Sequences do not overtake each other: behind one that found too few free pages every later one that needs a page
 * is refused too, whatever is free (with 5 free pages and needs of 6, 1 and 1 none is served), while those that need
 * no page are served.  So what must not wait, such as decode rows, comes before long prompts.  A sequence refused for
 * another reason holds nothing back.
 * No page id or length makes the call access anything outside the buffers.
 * seqs < 2^24, table_width * page_size < 2^30, tokens < 2^30 (FP4_ERR_SHAPE). */
fp4_status kv_pages_extend(const fp4_kv_pages *pool, int32_t *block_table, int64_t seqs, int64_t table_width,
                           int64_t table_stride, const int32_t *seq_lens, const int32_t *new_lens, int64_t tokens,
                           int32_t *lens_out, int32_t *state_out, int64_t *slots, int32_t *positions,
                           int32_t *cu_q, int32_t *cu_k, void *ws, size_t ws_bytes, hipStream_t stream);

/* Workspace bytes of kv_pages_collect (0: ws may be null). */
size_t kv_pages_collect_workspace(int64_t pages, int64_t seqs, int64_t table_width);

/* The free list anew: every page that no row holds in its first ceil(seq_lens[b] / page_size)
 * entries, in ascending order; state[0] is their number, entries past it are left.  So the pages of a
 * sequence that ended (its length set to 0), of dropped beams or of a shortened sequence come
 * back; a page held by several rows stays held.  Entries outside [0, pages) are passed over.
 * A page that no row of THIS table holds is free afterwards and is dealt again, so every holder of the pool's pages has to
 * stand in the one table: batches that share a pool are views of its rows, and a prompt kept for later use has a row of
 * its own there. */
fp4_status kv_pages_collect(const fp4_kv_pages *pool, const int32_t *block_table, int64_t seqs, int64_t table_width,
                            int64_t table_stride, const int32_t *seq_lens, void *ws, size_t ws_bytes,
                            hipStream_t stream);

/* Block tables of beams after a selection: row j of a group of `beams` rows takes the row of
 * its parent.
 *  block_table, out device int32 [batch * beams][stride]; out may be block_table itself (with the same
 *         stride; another overlap is not allowed).
 *  seq_lens int32 [batch * beams]; the rows of a group have the same length (below where they do not).
 *  parents int32 [batch * beams], each in [0, beams) (another value: the row keeps its own).
 *  copies int32 [batch * beams][3], out: {source page, destination page, tokens}, or
 *         {-1, -1, 0}.
 * Full pages are shared by the rows that hold them.  A partly filled page belongs to one row
 * (as kv_pages_extend deals them): a parent's first child keeps it, each further child gets
 * the partly filled page of a row that has no child, into which the parent's tokens have to be copied
 * (kv_cache_copy, once for each layer's cache).  Pages that no row holds any more come back with
 * kv_pages_collect.  Entries past a row's pages are left as they are.
 * Where the lengths differ (the pool ran out under some rows of a group) the group's tokens are lost, but no
 * other sequence's: a child whose spare row has no partly filled page there gets entry -1 and no copy, and
 * entries that a row's length covers but its parent's does not become -1.
 * beams <= 64; batch * ceil(table_width / 256) < 2^24 (FP4_ERR_SHAPE). */
fp4_status kv_pages_reorder(const int32_t *block_table, int64_t batch, int64_t beams, int64_t table_width,
                            int64_t table_stride, const int32_t *seq_lens, const int32_t *parents,
                            int64_t page_size, int32_t *out, int64_t out_stride, int32_t *copies,
                            hipStream_t stream);

/* For each of n records of `copies` (device int32 [n][3]) the first `tokens` tokens of the source page
 * are copied into the destination page: keys and values, codes and scale bytes, of all heads.  Records with
 * an id outside the cache or no tokens are skipped.  No page may be the destination of two records, or of one
 * and the source of another.  n * kv_heads < 2^23 (FP4_ERR_SHAPE); n == 0 returns FP4_OK. */
fp4_status kv_cache_copy(const fp4_kv_cache *cache, const int32_t *copies, int64_t n, hipStream_t stream);

/* Workspace bytes of beam_select. */
size_t beam_select_workspace(int64_t batch, int64_t beams, int64_t vocab, int64_t k, fp4_dtype xt);

/* Beam search's selection: for each of `batch` groups the k best of all beams' continuations,
 *   total(i, v) = score_i + logit_iv - log sum_u exp(logit_iu),
 * best first, equal ones by beam, then token (of one beam's: the larger logit first, also where its score leaves no
 * difference of logits in 64 bits).
 *  logits [batch * beams][ld] fp32 or bf16 (xt), ld >= vocab, any alignment of an element.
 *  scores fp32 [batch * beams], finite, or -infinity (NaN counts as such): the beam offers nothing.
 *  done   optional uint8 [batch * beams]: nonzero: the beam has ended and offers one
 *         continuation, end_token at its own score; its logits are not read.
 *  out_scores fp32, out_parents (the beam within its group) and out_tokens int32, [batch][k];
 *         out_scores may be scores (k == beams).
 * Totals of -infinity (masked tokens, beams that offer nothing; a row that holds a NaN or +infinity counts as
 * such) come last, in the order of beam and token, so that every place names a beam and a token.
 *  ws     beam_select_workspace() bytes, 16-byte aligned.
 * Totals are compared in 64 bits.  A row's sum is within 2^-18 relative: totals of two beams nearer than 2^-17 may stand
 * in either order, those of one beam always stand in the order of its logits.  1 <= k <= 64,
 * k <= beams * vocab, beams <= 64, beams * vocab <= 2^30, 0 <= end_token < vocab, batch < 2^21,
 * batch * beams * ceil(vocab / 4096) < 2^24 (FP4_ERR_SHAPE). */
fp4_status beam_select(const void *logits, fp4_dtype xt, int64_t batch, int64_t beams, int64_t vocab, int64_t ld,
                       const float *scores, const uint8_t *done, int64_t end_token, int64_t k, float *out_scores,
                       int32_t *out_parents, int32_t *out_tokens, void *ws, size_t ws_bytes, hipStream_t stream);

/* ---------------------------------------------------------- measurement --
 * fp4blk_read_ceiling: reads `bytes` bytes at `buf` once, with `grid`
 * workgroups of 512 threads striding over 16-byte words, and computes nothing
 * from them.  Its duration is the reference for the decode GEMV, which streams
 * its weight exactly once per call and is therefore bound by memory bandwidth
 * (edge-FP4 article, eefocus.com, section on the trade-offs of compute, memory
 * and precision).  A measurement aid, not part of the quantization path.
 * buf: device, 16-byte aligned; bytes: > 0, a multiple of 16; grid: 1..65535;
 * sink: device uint32, written only in the (practically never taken) case that
 * the XOR of all words equals a fixed constant.  FP4_ERR_NULL / _SHAPE /
 * _LAYOUT on bad arguments, nothing launched. */
fp4_status fp4blk_read_ceiling(const void *buf, size_t bytes, int grid, uint32_t *sink, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP4BLK_H */
