// abi.hip -- the extern "C" entry points of libfp4blk: argument validation,
// workspace layout and dispatch to the kernels.  Validation happens on the host
// before anything is launched, so an error leaves every output untouched.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>

#include "fp4blk.h"
#include "internal.h"

using namespace fp4k;

namespace {

constexpr int kMaxDevices = 64;
std::atomic<int> g_dev_state[kMaxDevices];  // 0 unknown, 1 gfx950, 2 other

fp4_status check_device()
{
    int dev = 0;
    int count = 0;
    if (hipGetDevice(&dev) == hipSuccess && dev >= 0 && dev < kMaxDevices &&
        g_dev_state[dev].load(std::memory_order_relaxed) == 1)
        return FP4_OK;  // seen before
    if (hipGetDeviceCount(&count) != hipSuccess || count <= 0) {
        (void)hipGetLastError();
        return FP4_ERR_NO_DEVICE;
    }
    if (hipGetDevice(&dev) != hipSuccess) return FP4_ERR_NO_DEVICE;
    if (dev < 0 || dev >= kMaxDevices) return FP4_ERR_UNSUPPORTED_DEVICE;
    int st = g_dev_state[dev].load(std::memory_order_relaxed);
    if (st == 0) {
        hipDeviceProp_t p;
        if (hipGetDeviceProperties(&p, dev) != hipSuccess) return FP4_ERR_HIP;
        st = std::strncmp(p.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        g_dev_state[dev].store(st, std::memory_order_relaxed);
    }
    return st == 1 ? FP4_OK : FP4_ERR_UNSUPPORTED_DEVICE;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t dsize(fp4_dtype t) { return t == FP4_F32 ? 4 : 2; }

bool valid_dtype(int t) { return t == FP4_F32 || t == FP4_BF16; }

// Kernels that address an operand with 32-bit buffer offsets take operands under
// 2 GiB; the entry points check this on the host, before anything is launched.
constexpr int64_t k2GiB = int64_t(1) << 31;

// M rows and N rows of row_bytes each both stay under 2 GiB
bool codes_under_2gib(int64_t M, int64_t N, int64_t row_bytes)
{
    return M * row_bytes < k2GiB && N * row_bytes < k2GiB;
}

// rows x cols input with leading dimension ld (elements of size es): rows stay
// 16-byte aligned when the base is and ld * es is a multiple of 16.
fp4_status check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, size_t es)
{
    if (!p) return FP4_ERR_NULL;
    if (rows <= 0 || cols <= 0) return FP4_ERR_SHAPE;
    if (ld < cols) return FP4_ERR_LAYOUT;
    if (!aligned16(p) || ((uint64_t)ld * es) % 16 != 0) return FP4_ERR_LAYOUT;
    return FP4_OK;
}

// packed operand (codes, scales): codes rows are cols/2 bytes, scale rows
// cols/block bytes; base pointers 16-byte aligned.
fp4_status check_packed(const uint8_t *codes, const uint8_t *scales)
{
    if (!codes || !scales) return FP4_ERR_NULL;
    if (!aligned16(codes) || !aligned16(scales)) return FP4_ERR_LAYOUT;
    return FP4_OK;
}

#define FP4_TRY(expr)                          \
    do {                                       \
        const fp4_status _s = (expr);          \
        if (_s != FP4_OK) return _s;           \
    } while (0)

}  // namespace

extern "C" {

const char *fp4_status_str(int s)
{
    switch (s) {
    case FP4_OK: return "FP4_OK";
    case FP4_ERR_NULL: return "FP4_ERR_NULL: a required pointer is null";
    case FP4_ERR_SHAPE: return "FP4_ERR_SHAPE: size <= 0, too large, or not a whole number of blocks";
    case FP4_ERR_LAYOUT: return "FP4_ERR_LAYOUT: leading dimension too small or pointer/row not 16-byte aligned";
    case FP4_ERR_DTYPE: return "FP4_ERR_DTYPE: unknown dtype, scale mode or MX rule";
    case FP4_ERR_WORKSPACE: return "FP4_ERR_WORKSPACE: workspace null or too small";
    case FP4_ERR_NO_DEVICE: return "FP4_ERR_NO_DEVICE: no HIP device visible";
    case FP4_ERR_UNSUPPORTED_DEVICE: return "FP4_ERR_UNSUPPORTED_DEVICE: current device is not gfx950";
    case FP4_ERR_HIP: return "FP4_ERR_HIP: a HIP call or kernel launch failed";
    default: return "unknown fp4_status";
    }
}

int fp4blk_version(void) { return 10000; }

fp4_status fp4blk_check_device(void) { return check_device(); }

fp4_status fp4blk_read_ceiling(const void *buf, size_t bytes, int grid, uint32_t *sink, hipStream_t stream)
{
    if (!buf || !sink) return FP4_ERR_NULL;
    if (bytes == 0 || bytes % 16 != 0 || grid <= 0 || grid > 65535) return FP4_ERR_SHAPE;
    if (!aligned16(buf)) return FP4_ERR_LAYOUT;
    FP4_TRY(check_device());
    return launch_read_ceiling(buf, bytes, grid, sink, stream);
}

// ------------------------------------------------------------------ NVFP4 --

size_t nvfp4_quantize_workspace(int64_t rows, int64_t cols, fp4_scale_mode mode)
{
    (void)rows;
    (void)cols;
    return mode == FP4_SCALE_PER_TENSOR ? kAmaxPartials * sizeof(float) : 0;
}

fp4_status nvfp4_quantize(const void *x, fp4_dtype xt, int64_t rows, int64_t cols, int64_t ldx,
                          uint8_t *codes, uint8_t *scales, float *tscale, fp4_scale_mode mode,
                          void *ws, size_t ws_bytes, int32_t *nonfinite, hipStream_t stream)
{
    if (!valid_dtype(xt) || (mode != FP4_SCALE_PER_TENSOR && mode != FP4_SCALE_PER_ROW))
        return FP4_ERR_DTYPE;
    FP4_TRY(check_matrix(x, rows, cols, ldx, dsize(xt)));
    if (cols % 16 != 0) return FP4_ERR_SHAPE;
    if (rows * cols > kMaxFlatElems) return FP4_ERR_SHAPE;
    if (!tscale) return FP4_ERR_NULL;
    FP4_TRY(check_packed(codes, scales));
    if (mode == FP4_SCALE_PER_TENSOR &&
        (!ws || ws_bytes < nvfp4_quantize_workspace(rows, cols, mode)))
        return FP4_ERR_WORKSPACE;
    FP4_TRY(check_device());
    return launch_nvfp4_quantize(x, xt, rows, cols, ldx, codes, scales, tscale, mode, ws, nonfinite,
                                 stream);
}

fp4_status nvfp4_dequantize(const uint8_t *codes, const uint8_t *scales, const float *tscale,
                            fp4_scale_mode mode, int64_t rows, int64_t cols, void *y,
                            fp4_dtype yt, int64_t ldy, hipStream_t stream)
{
    if (!valid_dtype(yt) || (mode != FP4_SCALE_PER_TENSOR && mode != FP4_SCALE_PER_ROW))
        return FP4_ERR_DTYPE;
    FP4_TRY(check_matrix(y, rows, cols, ldy, dsize(yt)));
    if (cols % 16 != 0) return FP4_ERR_SHAPE;
    if (rows * cols > kMaxFlatElems) return FP4_ERR_SHAPE;
    if (!tscale) return FP4_ERR_NULL;
    FP4_TRY(check_packed(codes, scales));
    FP4_TRY(check_device());
    return launch_nvfp4_dequantize(codes, scales, tscale, mode, rows, cols, y, yt, ldy, stream);
}

static fp4_status check_gemm_common(int64_t M, int64_t K, int64_t N, int kblock, const void *c,
                                    fp4_dtype ct, int64_t ldc)
{
    if (!valid_dtype(ct)) return FP4_ERR_DTYPE;
    if (M <= 0 || N <= 0 || K <= 0 || K % kblock != 0) return FP4_ERR_SHAPE;
    if (M > INT32_MAX / 2 || N > INT32_MAX / 2 || K > INT32_MAX / 2) return FP4_ERR_SHAPE;
    if (!c) return FP4_ERR_NULL;
    if (ldc < N) return FP4_ERR_LAYOUT;
    return FP4_OK;
}

fp4_status gemm_w4a16(const void *a, int64_t M, int64_t K, int64_t lda, const uint8_t *w_codes,
                      const uint8_t *w_scales, const float *w_tscale, int64_t N, void *c,
                      fp4_dtype ct, int64_t ldc, hipStream_t stream)
{
    FP4_TRY(check_gemm_common(M, K, N, 16, c, ct, ldc));
    FP4_TRY(check_matrix(a, M, K, lda, 2));
    FP4_TRY(check_packed(w_codes, w_scales));
    if (!w_tscale) return FP4_ERR_NULL;
    FP4_TRY(check_device());
    NvGemmArgs g{};
    g.a = reinterpret_cast<const uint16_t *>(a);
    g.lda = lda;
    g.w_codes = w_codes;
    g.w_scales = w_scales;
    g.w_tscale = w_tscale;
    g.M = M;
    g.N = N;
    g.K = K;
    g.c = c;
    g.c_bf16 = ct == FP4_BF16;
    g.ldc = ldc;
    return launch_nvfp4_gemm(g, stream);
}

fp4_status nvfp4_pack_decode(const uint8_t *codes, const uint8_t *scales, int64_t N, int64_t K,
                             uint8_t *codes_p, uint8_t *scales_p, hipStream_t stream)
{
    if (N <= 0 || K <= 0 || K % 128 != 0 || N > INT32_MAX / 2 || K > INT32_MAX / 2) return FP4_ERR_SHAPE;
    FP4_TRY(check_packed(codes, scales));
    FP4_TRY(check_packed(codes_p, scales_p));
    FP4_TRY(check_device());
    return launch_pack_decode(codes, scales, N, K, codes_p, scales_p, false, stream);
}

namespace {

// Both kernels behind the decode-layout entry points address A and the weight
// with 32-bit byte offsets (the GEMV's buffer descriptors hold 32-bit sizes, and
// its out-of-range offset 2^31 must lie past every operand): A's bytes up to its
// last element and the weight's code bytes stay below 2^31 for every M.
fp4_status check_decode_limits(int64_t M, int64_t K, int64_t lda, int64_t N)
{
    if ((M - 1) * lda * 2 + K * 2 >= k2GiB || M * lda * 2 >= k2GiB) return FP4_ERR_SHAPE;
    if (N * (K / 2) >= k2GiB) return FP4_ERR_SHAPE;
    return FP4_OK;
}

// M > 16 on a decode-layout weight: the prefill ring kernel reading that layout
fp4_status w4a16_seg_prefill(const void *a, int64_t M, int64_t K, int64_t lda, const uint8_t *w_codes_p,
                             const uint8_t *w_scales_p, const float *w_tscale, int64_t N, void *c, fp4_dtype ct,
                             int64_t ldc, bool mx, hipStream_t stream)
{
    NvGemmArgs g{};
    g.a = reinterpret_cast<const uint16_t *>(a);
    g.lda = lda;
    g.w_codes = w_codes_p;
    g.w_scales = w_scales_p;
    g.w_tscale = w_tscale;
    g.M = M;
    g.N = N;
    g.K = K;
    g.c = c;
    g.c_bf16 = ct == FP4_BF16;
    g.ldc = ldc;
    g.w_seg = 1;
    g.w_rows = N;
    g.w_row0 = 0;
    return launch_gemm_w4a16_seg(g, mx, stream);
}

}  // namespace

fp4_status gemm_w4a16_decode(const void *a, int64_t M, int64_t K, int64_t lda, const uint8_t *w_codes_p,
                             const uint8_t *w_scales_p, const float *w_tscale, int64_t N, void *c,
                             fp4_dtype ct, int64_t ldc, hipStream_t stream)
{
    FP4_TRY(check_gemm_common(M, K, N, 128, c, ct, ldc));
    FP4_TRY(check_matrix(a, M, K, lda, 2));
    FP4_TRY(check_decode_limits(M, K, lda, N));
    FP4_TRY(check_packed(w_codes_p, w_scales_p));
    if (!w_tscale) return FP4_ERR_NULL;
    FP4_TRY(check_device());
    if (M > 16) return w4a16_seg_prefill(a, M, K, lda, w_codes_p, w_scales_p, w_tscale, N, c, ct, ldc, false, stream);
    GemvArgs g{};
    g.a = reinterpret_cast<const uint16_t *>(a);
    g.lda = lda;
    g.w_codes = w_codes_p;
    g.w_scales = w_scales_p;
    g.w_tscale = w_tscale;
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)K;
    g.c = c;
    g.c_bf16 = ct == FP4_BF16;
    g.ldc = ldc;
    return launch_gemv_decode(g, stream);
}

fp4_status mxfp4_pack_decode(const uint8_t *codes, const uint8_t *scales, int64_t N, int64_t K,
                             uint8_t *codes_p, uint8_t *scales_p, hipStream_t stream)
{
    if (N <= 0 || K <= 0 || K % 128 != 0 || N > INT32_MAX / 2 || K > INT32_MAX / 2) return FP4_ERR_SHAPE;
    FP4_TRY(check_packed(codes, scales));
    FP4_TRY(check_packed(codes_p, scales_p));
    FP4_TRY(check_device());
    return launch_pack_decode(codes, scales, N, K, codes_p, scales_p, true, stream);
}

fp4_status mxfp4_gemm_w4a16_decode(const void *a, int64_t M, int64_t K, int64_t lda, const uint8_t *w_codes_p,
                                   const uint8_t *w_scales_p, int64_t N, void *c, fp4_dtype ct, int64_t ldc,
                                   hipStream_t stream)
{
    FP4_TRY(check_gemm_common(M, K, N, 128, c, ct, ldc));
    FP4_TRY(check_matrix(a, M, K, lda, 2));
    FP4_TRY(check_decode_limits(M, K, lda, N));
    FP4_TRY(check_packed(w_codes_p, w_scales_p));
    FP4_TRY(check_device());
    if (M > 16) return w4a16_seg_prefill(a, M, K, lda, w_codes_p, w_scales_p, nullptr, N, c, ct, ldc, true, stream);
    GemvArgs g{};
    g.a = reinterpret_cast<const uint16_t *>(a);
    g.lda = lda;
    g.w_codes = w_codes_p;
    g.w_scales = w_scales_p;
    g.w_tscale = nullptr;
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)K;
    g.mx = 1;
    g.c = c;
    g.c_bf16 = ct == FP4_BF16;
    g.ldc = ldc;
    return launch_gemv_decode(g, stream);
}

fp4_status mxfp4_gemm_w4a16(const void *a, int64_t M, int64_t K, int64_t lda, const uint8_t *w_codes,
                            const uint8_t *w_scales, int64_t N, void *c, fp4_dtype ct, int64_t ldc,
                            hipStream_t stream)
{
    FP4_TRY(check_gemm_common(M, K, N, 128, c, ct, ldc));
    FP4_TRY(check_matrix(a, M, K, lda, 2));
    FP4_TRY(check_packed(w_codes, w_scales));
    FP4_TRY(check_device());
    NvGemmArgs g{};
    g.a = reinterpret_cast<const uint16_t *>(a);
    g.lda = lda;
    g.w_codes = w_codes;
    g.w_scales = w_scales;
    g.w_tscale = nullptr;
    g.M = M;
    g.N = N;
    g.K = K;
    g.c = c;
    g.c_bf16 = ct == FP4_BF16;
    g.ldc = ldc;
    return launch_mxfp4_gemm_w4a16(g, stream);
}

void gemm_w4a4_workspace_offsets(int64_t M, int64_t K, size_t *codes_off, size_t *scales_off,
                                 size_t *tscale_off)
{
    const size_t cb = align256((size_t)M * (size_t)(K / 2));
    const size_t sb = align256((size_t)M * (size_t)(K / 16));
    if (codes_off) *codes_off = 0;
    if (scales_off) *scales_off = cb;
    if (tscale_off) *tscale_off = cb + sb;
}

size_t gemm_w4a4_workspace(int64_t M, int64_t K, fp4_scale_mode a_mode)
{
    if (M <= 0 || K <= 0) return 0;
    size_t t;
    gemm_w4a4_workspace_offsets(M, K, nullptr, nullptr, &t);
    const size_t ts = align256((size_t)(a_mode == FP4_SCALE_PER_ROW ? M : 1) * sizeof(float));
    // the per-tensor amax partials follow the tensor scale
    const size_t amax = a_mode == FP4_SCALE_PER_TENSOR ? kAmaxPartials * sizeof(float) : 0;
    return t + ts + amax;
}

namespace {

// the GEMM half of the NVFP4 W4A4 forms, arguments checked (w_seg: W in the decode layout)
fp4_status w4a4_launch(const uint8_t *a_codes, const uint8_t *a_scales, const float *a_tscale, fp4_scale_mode a_mode,
                       int64_t M, int64_t K, const uint8_t *w_codes, const uint8_t *w_scales, const float *w_tscale,
                       int64_t N, void *c, fp4_dtype ct, int64_t ldc, bool w_seg, hipStream_t stream)
{
    NvGemmArgs g{};
    g.a_codes = a_codes;
    g.a_scales = a_scales;
    g.a_tscale = a_tscale;
    g.a_per_row = a_mode == FP4_SCALE_PER_ROW;
    g.w_codes = w_codes;
    g.w_scales = w_scales;
    g.w_tscale = w_tscale;
    g.M = M;
    g.N = N;
    g.K = K;
    g.c = c;
    g.c_bf16 = ct == FP4_BF16;
    g.ldc = ldc;
    if (!w_seg) return launch_nvfp4_gemm(g, stream);
    g.w_seg = 1;
    g.w_rows = N;
    g.w_row0 = 0;
    return launch_gemm_w4a4_seg(g, stream);
}

fp4_status w4a4_prequant(const uint8_t *a_codes, const uint8_t *a_scales, const float *a_tscale, fp4_scale_mode a_mode,
                         int64_t M, int64_t K, const uint8_t *w_codes, const uint8_t *w_scales, const float *w_tscale,
                         int64_t N, void *c, fp4_dtype ct, int64_t ldc, bool w_seg, hipStream_t stream)
{
    if (a_mode != FP4_SCALE_PER_TENSOR && a_mode != FP4_SCALE_PER_ROW) return FP4_ERR_DTYPE;
    FP4_TRY(check_gemm_common(M, K, N, w_seg ? 128 : 16, c, ct, ldc));
    FP4_TRY(check_packed(a_codes, a_scales));
    FP4_TRY(check_packed(w_codes, w_scales));
    if (!a_tscale || !w_tscale) return FP4_ERR_NULL;
    if (w_seg && !codes_under_2gib(M, N, K / 2)) return FP4_ERR_SHAPE;
    FP4_TRY(check_device());
    return w4a4_launch(a_codes, a_scales, a_tscale, a_mode, M, K, w_codes, w_scales, w_tscale, N, c, ct, ldc, w_seg,
                       stream);
}

fp4_status w4a4_full(const void *a, int64_t M, int64_t K, int64_t lda, fp4_scale_mode a_mode, const uint8_t *w_codes,
                     const uint8_t *w_scales, const float *w_tscale, int64_t N, void *c, fp4_dtype ct, int64_t ldc,
                     void *ws, size_t ws_bytes, bool w_seg, hipStream_t stream)
{
    if (a_mode != FP4_SCALE_PER_TENSOR && a_mode != FP4_SCALE_PER_ROW) return FP4_ERR_DTYPE;
    FP4_TRY(check_gemm_common(M, K, N, w_seg ? 128 : 16, c, ct, ldc));
    FP4_TRY(check_matrix(a, M, K, lda, 2));
    if (M * K > kMaxFlatElems) return FP4_ERR_SHAPE;
    FP4_TRY(check_packed(w_codes, w_scales));
    if (!w_tscale) return FP4_ERR_NULL;
    if (!ws || !aligned16(ws) || ws_bytes < gemm_w4a4_workspace(M, K, a_mode))
        return FP4_ERR_WORKSPACE;
    if (w_seg && !codes_under_2gib(M, N, K / 2)) return FP4_ERR_SHAPE;  // before A is quantized
    FP4_TRY(check_device());
    size_t co, so, to;
    gemm_w4a4_workspace_offsets(M, K, &co, &so, &to);
    uint8_t *base = reinterpret_cast<uint8_t *>(ws);
    uint8_t *ac = base + co;
    uint8_t *as = base + so;
    float *at = reinterpret_cast<float *>(base + to);
    void *amax_ws = base + to + align256((size_t)(a_mode == FP4_SCALE_PER_ROW ? M : 1) * sizeof(float));
    FP4_TRY(launch_nvfp4_quantize(a, FP4_BF16, M, K, lda, ac, as, at, a_mode, amax_ws, nullptr,
                                  stream));
    return w4a4_launch(ac, as, at, a_mode, M, K, w_codes, w_scales, w_tscale, N, c, ct, ldc, w_seg, stream);
}

}  // namespace

fp4_status gemm_nvfp4_w4a4_prequant(const uint8_t *a_codes, const uint8_t *a_scales,
                                    const float *a_tscale, fp4_scale_mode a_mode, int64_t M,
                                    int64_t K, const uint8_t *w_codes, const uint8_t *w_scales,
                                    const float *w_tscale, int64_t N, void *c, fp4_dtype ct,
                                    int64_t ldc, hipStream_t stream)
{
    return w4a4_prequant(a_codes, a_scales, a_tscale, a_mode, M, K, w_codes, w_scales, w_tscale, N, c, ct, ldc, false,
                         stream);
}

fp4_status gemm_w4a4(const void *a, int64_t M, int64_t K, int64_t lda, fp4_scale_mode a_mode,
                     const uint8_t *w_codes, const uint8_t *w_scales, const float *w_tscale,
                     int64_t N, void *c, fp4_dtype ct, int64_t ldc, void *ws, size_t ws_bytes,
                     hipStream_t stream)
{
    return w4a4_full(a, M, K, lda, a_mode, w_codes, w_scales, w_tscale, N, c, ct, ldc, ws, ws_bytes, false, stream);
}

fp4_status gemm_nvfp4_w4a4_prequant_seg(const uint8_t *a_codes, const uint8_t *a_scales, const float *a_tscale,
                                        fp4_scale_mode a_mode, int64_t M, int64_t K, const uint8_t *w_codes_p,
                                        const uint8_t *w_scales_p, const float *w_tscale, int64_t N, void *c,
                                        fp4_dtype ct, int64_t ldc, hipStream_t stream)
{
    return w4a4_prequant(a_codes, a_scales, a_tscale, a_mode, M, K, w_codes_p, w_scales_p, w_tscale, N, c, ct, ldc,
                         true, stream);
}

fp4_status gemm_w4a4_seg(const void *a, int64_t M, int64_t K, int64_t lda, fp4_scale_mode a_mode,
                         const uint8_t *w_codes_p, const uint8_t *w_scales_p, const float *w_tscale, int64_t N,
                         void *c, fp4_dtype ct, int64_t ldc, void *ws, size_t ws_bytes, hipStream_t stream)
{
    return w4a4_full(a, M, K, lda, a_mode, w_codes_p, w_scales_p, w_tscale, N, c, ct, ldc, ws, ws_bytes, true, stream);
}

}  // extern "C"

// ------------------------------------------------ W4A4 without allocation --
//
// gemm_w4a4_noalloc keeps A's packed form in `scratch`, a device array of the
// library itself, instead of a caller's workspace.  Each device holds its own
// copy from the time the library's code is loaded on it until the process ends.
// In host code `scratch` names a host-side stand-in, never device memory: its
// device address is looked up once per device (hipGetSymbolAddress, with that
// device current) and only that address is passed to kernels.  Nothing in it
// needs clearing between calls: the quantizer writes every byte the GEMM reads
// (codes, scales, tensor scales and, per tensor, all amax partials it reduces).

namespace {

constexpr size_t kNoallocScratchBytes = size_t(32) << 20;

static __device__ __align__(256) uint8_t scratch[kNoallocScratchBytes];

std::atomic<uintptr_t> g_scratch_addr[kMaxDevices];  // 0 until looked up on that device

// The device address of the current device's `scratch`, or null on failure.
void *scratch_on_current_device()
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    uintptr_t p = g_scratch_addr[dev].load(std::memory_order_acquire);
    if (!p) {
        void *q = nullptr;
        if (hipGetSymbolAddress(&q, HIP_SYMBOL(scratch)) != hipSuccess || !q) {
            (void)hipGetLastError();
            return nullptr;
        }
        p = reinterpret_cast<uintptr_t>(q);
        g_scratch_addr[dev].store(p, std::memory_order_release);  // racing first calls store the same address
    }
    return reinterpret_cast<void *>(p);
}

}  // namespace

extern "C" {

fp4_status gemm_w4a4_noalloc(const void *a, int64_t M, int64_t K, int64_t lda, fp4_scale_mode a_mode,
                             const uint8_t *w_codes, const uint8_t *w_scales, const float *w_tscale, int64_t N,
                             void *c, fp4_dtype ct, int64_t ldc, hipStream_t stream)
{
    if (a_mode != FP4_SCALE_PER_TENSOR && a_mode != FP4_SCALE_PER_ROW) return FP4_ERR_DTYPE;
    FP4_TRY(check_gemm_common(M, K, N, 16, c, ct, ldc));
    FP4_TRY(check_matrix(a, M, K, lda, 2));
    if (M * K > kMaxFlatElems) return FP4_ERR_SHAPE;
    FP4_TRY(check_packed(w_codes, w_scales));
    if (!w_tscale) return FP4_ERR_NULL;
    if (gemm_w4a4_workspace(M, K, a_mode) > kNoallocScratchBytes) return FP4_ERR_WORKSPACE;
    FP4_TRY(check_device());
    void *ws = scratch_on_current_device();
    if (!ws) return FP4_ERR_HIP;
    return w4a4_full(a, M, K, lda, a_mode, w_codes, w_scales, w_tscale, N, c, ct, ldc, ws, kNoallocScratchBytes, false,
                     stream);
}

// ------------------------------------------------------------------ MXFP4 --

fp4_status mxfp4_quantize(const void *x, fp4_dtype xt, int64_t rows, int64_t cols, int64_t ldx,
                          uint8_t *codes, uint8_t *scales, fp4_mx_rule rule, int32_t *nonfinite,
                          hipStream_t stream)
{
    if (!valid_dtype(xt) || (rule != FP4_MX_OCP_FLOOR && rule != FP4_MX_CEIL)) return FP4_ERR_DTYPE;
    FP4_TRY(check_matrix(x, rows, cols, ldx, dsize(xt)));
    if (cols % 32 != 0) return FP4_ERR_SHAPE;
    if (rows * cols > kMaxFlatElems) return FP4_ERR_SHAPE;
    FP4_TRY(check_packed(codes, scales));
    FP4_TRY(check_device());
    return launch_mxfp4_quantize(x, xt, rows, cols, ldx, codes, scales, rule, nonfinite, stream);
}

fp4_status mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                            int64_t cols, void *y, fp4_dtype yt, int64_t ldy, hipStream_t stream)
{
    if (!valid_dtype(yt)) return FP4_ERR_DTYPE;
    FP4_TRY(check_matrix(y, rows, cols, ldy, dsize(yt)));
    if (cols % 32 != 0) return FP4_ERR_SHAPE;
    if (rows * cols > kMaxFlatElems) return FP4_ERR_SHAPE;
    FP4_TRY(check_packed(codes, scales));
    FP4_TRY(check_device());
    return launch_mxfp4_dequantize(codes, scales, rows, cols, y, yt, ldy, stream);
}

size_t mxfp4_gemm_w4a4_workspace(int64_t M, int64_t K)
{
    if (M <= 0 || K <= 0) return 0;
    return align256((size_t)M * (size_t)(K / 2)) + align256((size_t)M * (size_t)(K / 32));
}

fp4_status mxfp4_gemm_prequant(const uint8_t *a_codes, const uint8_t *a_scales, int64_t M,
                               int64_t K, const uint8_t *w_codes, const uint8_t *w_scales,
                               int64_t N, void *c, fp4_dtype ct, int64_t ldc, hipStream_t stream)
{
    FP4_TRY(check_gemm_common(M, K, N, 32, c, ct, ldc));
    FP4_TRY(check_packed(a_codes, a_scales));
    FP4_TRY(check_packed(w_codes, w_scales));
    FP4_TRY(check_device());
    MxGemmArgs g{};
    g.a_codes = a_codes;
    g.a_scales = a_scales;
    g.w_codes = w_codes;
    g.w_scales = w_scales;
    g.M = M;
    g.N = N;
    g.K = K;
    g.c = c;
    g.c_bf16 = ct == FP4_BF16;
    g.ldc = ldc;
    return launch_mxfp4_gemm(g, stream);
}

int mxfp4_gemm_w4a4_a_segment_major(int64_t M, int64_t N, int64_t K)
{
    return M > 0 && N > 0 && K > 0 && K % 128 == 0 && codes_under_2gib(M, N, K / 2) ? 1 : 0;
}

fp4_status mxfp4_gemm_w4a4(const void *a, int64_t M, int64_t K, int64_t lda, fp4_mx_rule rule,
                           const uint8_t *w_codes, const uint8_t *w_scales, int64_t N, void *c,
                           fp4_dtype ct, int64_t ldc, void *ws, size_t ws_bytes,
                           hipStream_t stream)
{
    if (rule != FP4_MX_OCP_FLOOR && rule != FP4_MX_CEIL) return FP4_ERR_DTYPE;
    FP4_TRY(check_gemm_common(M, K, N, 32, c, ct, ldc));
    FP4_TRY(check_matrix(a, M, K, lda, 2));
    if (M * K > kMaxFlatElems) return FP4_ERR_SHAPE;
    FP4_TRY(check_packed(w_codes, w_scales));
    if (!ws || !aligned16(ws) || ws_bytes < mxfp4_gemm_w4a4_workspace(M, K)) return FP4_ERR_WORKSPACE;
    FP4_TRY(check_device());
    uint8_t *ac = reinterpret_cast<uint8_t *>(ws);
    uint8_t *as = ac + align256((size_t)M * (size_t)(K / 2));
    // A's packed form lives only in the workspace, so its layout is this call's
    // choice: segment-major (each 256-row panel's 128-K segment one contiguous
    // 16 KiB run) whenever the segment kernel applies, with W read row-major by
    // the same kernel; the products and their order, and so C, are the same
    const bool seg = mxfp4_gemm_w4a4_a_segment_major(M, N, K) != 0;
    if (seg)
        FP4_TRY(launch_mxfp4_quantize_seg(a, FP4_BF16, M, K, lda, ac, as, rule, nullptr, stream));
    else
        FP4_TRY(launch_mxfp4_quantize(a, FP4_BF16, M, K, lda, ac, as, rule, nullptr, stream));
    MxGemmArgs g{};
    g.a_codes = ac;
    g.a_scales = as;
    g.w_codes = w_codes;
    g.w_scales = w_scales;
    g.M = M;
    g.N = N;
    g.K = K;
    g.c = c;
    g.c_bf16 = ct == FP4_BF16;
    g.ldc = ldc;
    return seg ? launch_mxfp4_gemm_seg_wrow(g, stream) : launch_mxfp4_gemm(g, stream);
}

// ------------------------------------------- MXFP4 W4A4, segment-major ----

size_t mxfp4_gemm_w4a4_seg_workspace(int64_t M, int64_t K)
{
    return mxfp4_gemm_w4a4_workspace(M, K);  // the same bytes, in the other order
}

fp4_status mxfp4_gemm_prequant_seg(const uint8_t *a_codes_p, const uint8_t *a_scales_p, int64_t M, int64_t K,
                                   const uint8_t *w_codes_p, const uint8_t *w_scales_p, int64_t N, void *c,
                                   fp4_dtype ct, int64_t ldc, hipStream_t stream)
{
    FP4_TRY(check_gemm_common(M, K, N, 128, c, ct, ldc));
    FP4_TRY(check_packed(a_codes_p, a_scales_p));
    FP4_TRY(check_packed(w_codes_p, w_scales_p));
    if (!codes_under_2gib(M, N, K / 2)) return FP4_ERR_SHAPE;
    FP4_TRY(check_device());
    MxGemmArgs g{};
    g.a_codes = a_codes_p;
    g.a_scales = a_scales_p;
    g.w_codes = w_codes_p;
    g.w_scales = w_scales_p;
    g.M = M;
    g.N = N;
    g.K = K;
    g.c = c;
    g.c_bf16 = ct == FP4_BF16;
    g.ldc = ldc;
    return launch_mxfp4_gemm_seg(g, stream);
}

fp4_status mxfp4_gemm_w4a4_seg(const void *a, int64_t M, int64_t K, int64_t lda, fp4_mx_rule rule,
                               const uint8_t *w_codes_p, const uint8_t *w_scales_p, int64_t N, void *c,
                               fp4_dtype ct, int64_t ldc, void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (rule != FP4_MX_OCP_FLOOR && rule != FP4_MX_CEIL) return FP4_ERR_DTYPE;
    FP4_TRY(check_gemm_common(M, K, N, 128, c, ct, ldc));
    FP4_TRY(check_matrix(a, M, K, lda, 2));
    if (M * K > kMaxFlatElems) return FP4_ERR_SHAPE;
    FP4_TRY(check_packed(w_codes_p, w_scales_p));
    if (!ws || !aligned16(ws) || ws_bytes < mxfp4_gemm_w4a4_seg_workspace(M, K)) return FP4_ERR_WORKSPACE;
    if (!codes_under_2gib(M, N, K / 2)) return FP4_ERR_SHAPE;  // before A is quantized
    FP4_TRY(check_device());
    uint8_t *ac = reinterpret_cast<uint8_t *>(ws);
    uint8_t *as = ac + align256((size_t)M * (size_t)(K / 2));
    FP4_TRY(launch_mxfp4_quantize_seg(a, FP4_BF16, M, K, lda, ac, as, rule, nullptr, stream));
    MxGemmArgs g{};
    g.a_codes = ac;
    g.a_scales = as;
    g.w_codes = w_codes_p;
    g.w_scales = w_scales_p;
    g.M = M;
    g.N = N;
    g.K = K;
    g.c = c;
    g.c_bf16 = ct == FP4_BF16;
    g.ldc = ldc;
    return launch_mxfp4_gemm_seg(g, stream);
}

// ------------------------------------------------------------------- W4A8 --

fp4_status mxfp8_quantize(const void *x, fp4_dtype xt, int64_t rows, int64_t cols, int64_t ldx,
                          uint8_t *codes, uint8_t *scales, fp4_mx_rule rule, int32_t *nonfinite,
                          hipStream_t stream)
{
    if (!valid_dtype(xt) || (rule != FP4_MX_OCP_FLOOR && rule != FP4_MX_CEIL)) return FP4_ERR_DTYPE;
    FP4_TRY(check_matrix(x, rows, cols, ldx, dsize(xt)));
    if (cols % 32 != 0) return FP4_ERR_SHAPE;
    if (rows * cols > kMaxFlatElems) return FP4_ERR_SHAPE;
    FP4_TRY(check_packed(codes, scales));
    FP4_TRY(check_device());
    return launch_mxfp8_quantize(x, xt, rows, cols, ldx, codes, scales, rule, nonfinite, stream);
}

size_t mxfp4_gemm_w4a8_workspace(int64_t M, int64_t K)
{
    if (M <= 0 || K <= 0) return 0;
    return align256((size_t)M * (size_t)K) + align256((size_t)M * (size_t)(K / 32));
}

namespace {

// the GEMM half of both W4A8 forms (w_seg: W segment-major)
fp4_status w4a8_gemm(const uint8_t *a_codes, const uint8_t *a_scales, int64_t M, int64_t K, const uint8_t *w_codes,
                     const uint8_t *w_scales, int64_t N, void *c, fp4_dtype ct, int64_t ldc, bool w_seg,
                     hipStream_t stream)
{
    FP4_TRY(check_gemm_common(M, K, N, 128, c, ct, ldc));
    FP4_TRY(check_packed(a_codes, a_scales));
    FP4_TRY(check_packed(w_codes, w_scales));
    if (M * K >= k2GiB || !codes_under_2gib(0, N, K / 2)) return FP4_ERR_SHAPE;
    FP4_TRY(check_device());
    MxGemmArgs g{};
    g.a_codes = a_codes;
    g.a_scales = a_scales;
    g.w_codes = w_codes;
    g.w_scales = w_scales;
    g.M = M;
    g.N = N;
    g.K = K;
    g.c = c;
    g.c_bf16 = ct == FP4_BF16;
    g.ldc = ldc;
    g.w_seg = w_seg ? 1 : 0;
    return launch_mxfp4_gemm_w4a8(g, stream);
}

fp4_status w4a8_full(const void *a, int64_t M, int64_t K, int64_t lda, fp4_mx_rule rule, const uint8_t *w_codes,
                     const uint8_t *w_scales, int64_t N, void *c, fp4_dtype ct, int64_t ldc, void *ws,
                     size_t ws_bytes, bool w_seg, hipStream_t stream)
{
    if (rule != FP4_MX_OCP_FLOOR && rule != FP4_MX_CEIL) return FP4_ERR_DTYPE;
    FP4_TRY(check_gemm_common(M, K, N, 128, c, ct, ldc));
    FP4_TRY(check_matrix(a, M, K, lda, 2));
    if (M * K > kMaxFlatElems) return FP4_ERR_SHAPE;
    FP4_TRY(check_packed(w_codes, w_scales));
    if (!ws || !aligned16(ws) || ws_bytes < mxfp4_gemm_w4a8_workspace(M, K)) return FP4_ERR_WORKSPACE;
    if (M * K >= k2GiB || !codes_under_2gib(0, N, K / 2)) return FP4_ERR_SHAPE;  // before A is quantized
    FP4_TRY(check_device());
    uint8_t *ac = reinterpret_cast<uint8_t *>(ws);
    uint8_t *as = ac + align256((size_t)M * (size_t)K);
    FP4_TRY(launch_mxfp8_quantize(a, FP4_BF16, M, K, lda, ac, as, rule, nullptr, stream));
    return w4a8_gemm(ac, as, M, K, w_codes, w_scales, N, c, ct, ldc, w_seg, stream);
}

}  // namespace

fp4_status mxfp4_gemm_w4a8_prequant(const uint8_t *a_codes, const uint8_t *a_scales, int64_t M, int64_t K,
                                    const uint8_t *w_codes, const uint8_t *w_scales, int64_t N, void *c,
                                    fp4_dtype ct, int64_t ldc, hipStream_t stream)
{
    return w4a8_gemm(a_codes, a_scales, M, K, w_codes, w_scales, N, c, ct, ldc, false, stream);
}

fp4_status mxfp4_gemm_w4a8(const void *a, int64_t M, int64_t K, int64_t lda, fp4_mx_rule rule,
                           const uint8_t *w_codes, const uint8_t *w_scales, int64_t N, void *c,
                           fp4_dtype ct, int64_t ldc, void *ws, size_t ws_bytes, hipStream_t stream)
{
    return w4a8_full(a, M, K, lda, rule, w_codes, w_scales, N, c, ct, ldc, ws, ws_bytes, false, stream);
}

fp4_status mxfp4_gemm_w4a8_prequant_seg(const uint8_t *a_codes, const uint8_t *a_scales, int64_t M, int64_t K,
                                        const uint8_t *w_codes_p, const uint8_t *w_scales_p, int64_t N, void *c,
                                        fp4_dtype ct, int64_t ldc, hipStream_t stream)
{
    return w4a8_gemm(a_codes, a_scales, M, K, w_codes_p, w_scales_p, N, c, ct, ldc, true, stream);
}

fp4_status mxfp4_gemm_w4a8_seg(const void *a, int64_t M, int64_t K, int64_t lda, fp4_mx_rule rule,
                               const uint8_t *w_codes_p, const uint8_t *w_scales_p, int64_t N, void *c,
                               fp4_dtype ct, int64_t ldc, void *ws, size_t ws_bytes, hipStream_t stream)
{
    return w4a8_full(a, M, K, lda, rule, w_codes_p, w_scales_p, N, c, ct, ldc, ws, ws_bytes, true, stream);
}

// ------------------------------------------------------- grouped (MoE) --

namespace {

constexpr int64_t kMaxGroups = 1 << 16;

// Arguments every grouped GEMM shares.  rows == 0 (no routed rows) is valid: once
// the sizes and group arguments check out, *empty is set and the caller returns
// FP4_OK without touching A, W or C (which may then be empty, even null).
fp4_status check_grouped(int64_t a_rows, int64_t K, const int32_t *row_index, const int32_t *group_offs,
                         int64_t groups, int64_t rows, int64_t N, int kblock, const void *c, fp4_dtype ct,
                         int64_t ldc, bool *empty)
{
    if (rows < 0) return FP4_ERR_SHAPE;
    if (groups <= 0 || groups > kMaxGroups) return FP4_ERR_SHAPE;
    if (!group_offs) return FP4_ERR_NULL;
    *empty = rows == 0;
    if (*empty) {
        if (!valid_dtype(ct)) return FP4_ERR_DTYPE;
        return N > 0 && K > 0 && K % kblock == 0 ? FP4_OK : FP4_ERR_SHAPE;
    }
    FP4_TRY(check_gemm_common(rows, K, N, kblock, c, ct, ldc));
    if (a_rows <= 0 || a_rows > INT32_MAX / 2) return FP4_ERR_SHAPE;
    if (!row_index && a_rows < rows) return FP4_ERR_SHAPE;
    return FP4_OK;
}

// The grouped kernel's own limits, checked here so that nothing (not even the
// W4A4 activation quantizer) is launched for a call the kernel would refuse:
// 32-bit byte offsets into A (its bf16 rows, or its packed codes for W4A4) and
// into one group's weight codes, and a grid below 2^31 workgroups.
fp4_status check_grouped_limits(int64_t a_rows, int64_t K, int64_t lda, bool a_fp4, int64_t groups,
                                int64_t rows, int64_t N)
{
    const int64_t a_bytes = a_fp4 ? a_rows * (K / 2) : a_rows * lda * 2;
    if (a_bytes >= k2GiB || N * (K / 2) >= k2GiB) return FP4_ERR_SHAPE;
    if (((rows + 127) / 128 + groups) * ((N + 255) / 256) >= k2GiB) return FP4_ERR_SHAPE;
    return FP4_OK;
}

NvGemmArgs grouped_args(int64_t a_rows, int64_t K, const int32_t *row_index, const int32_t *group_offs,
                        int64_t groups, int64_t rows, const uint8_t *w_codes, const uint8_t *w_scales,
                        const float *w_tscale, int64_t N, void *c, fp4_dtype ct, int64_t ldc)
{
    NvGemmArgs g{};
    g.w_codes = w_codes;
    g.w_scales = w_scales;
    g.w_tscale = w_tscale;
    g.M = rows;
    g.N = N;
    g.K = K;
    g.c = c;
    g.c_bf16 = ct == FP4_BF16;
    g.ldc = ldc;
    g.groups = (int)groups;
    g.group_offs = group_offs;
    g.row_index = row_index;
    g.a_rows = a_rows;
    return g;
}

}  // namespace

fp4_status nvfp4_grouped_gemm_w4a16(const void *a, int64_t a_rows, int64_t K, int64_t lda,
                                    const int32_t *row_index, const int32_t *group_offs, int64_t groups,
                                    int64_t rows, const uint8_t *w_codes, const uint8_t *w_scales,
                                    const float *w_tscale, int64_t N, void *c, fp4_dtype ct, int64_t ldc,
                                    hipStream_t stream)
{
    bool empty = false;
    FP4_TRY(check_grouped(a_rows, K, row_index, group_offs, groups, rows, N, 64, c, ct, ldc, &empty));
    if (empty) return FP4_OK;
    FP4_TRY(check_matrix(a, a_rows, K, lda, 2));
    FP4_TRY(check_grouped_limits(a_rows, K, lda, false, groups, rows, N));
    FP4_TRY(check_packed(w_codes, w_scales));
    if (!w_tscale) return FP4_ERR_NULL;
    FP4_TRY(check_device());
    NvGemmArgs g = grouped_args(a_rows, K, row_index, group_offs, groups, rows, w_codes, w_scales, w_tscale, N, c,
                                ct, ldc);
    g.a = reinterpret_cast<const uint16_t *>(a);
    g.lda = lda;
    return launch_grouped_gemm(g, 0, stream);
}

fp4_status mxfp4_grouped_gemm_w4a16(const void *a, int64_t a_rows, int64_t K, int64_t lda,
                                    const int32_t *row_index, const int32_t *group_offs, int64_t groups,
                                    int64_t rows, const uint8_t *w_codes, const uint8_t *w_scales, int64_t N,
                                    void *c, fp4_dtype ct, int64_t ldc, hipStream_t stream)
{
    bool empty = false;
    FP4_TRY(check_grouped(a_rows, K, row_index, group_offs, groups, rows, N, 128, c, ct, ldc, &empty));
    if (empty) return FP4_OK;
    FP4_TRY(check_matrix(a, a_rows, K, lda, 2));
    FP4_TRY(check_grouped_limits(a_rows, K, lda, false, groups, rows, N));
    FP4_TRY(check_packed(w_codes, w_scales));
    FP4_TRY(check_device());
    NvGemmArgs g = grouped_args(a_rows, K, row_index, group_offs, groups, rows, w_codes, w_scales, nullptr, N, c,
                                ct, ldc);
    g.a = reinterpret_cast<const uint16_t *>(a);
    g.lda = lda;
    return launch_grouped_gemm(g, 2, stream);
}

fp4_status nvfp4_grouped_gemm_w4a4_prequant(const uint8_t *a_codes, const uint8_t *a_scales,
                                            const float *a_tscale, int64_t a_rows, int64_t K,
                                            const int32_t *row_index, const int32_t *group_offs,
                                            int64_t groups, int64_t rows, const uint8_t *w_codes,
                                            const uint8_t *w_scales, const float *w_tscale, int64_t N,
                                            void *c, fp4_dtype ct, int64_t ldc, hipStream_t stream)
{
    bool empty = false;
    FP4_TRY(check_grouped(a_rows, K, row_index, group_offs, groups, rows, N, 64, c, ct, ldc, &empty));
    if (empty) return FP4_OK;
    FP4_TRY(check_grouped_limits(a_rows, K, K, true, groups, rows, N));
    FP4_TRY(check_packed(a_codes, a_scales));
    FP4_TRY(check_packed(w_codes, w_scales));
    if (!a_tscale || !w_tscale) return FP4_ERR_NULL;
    FP4_TRY(check_device());
    NvGemmArgs g = grouped_args(a_rows, K, row_index, group_offs, groups, rows, w_codes, w_scales, w_tscale, N, c,
                                ct, ldc);
    g.a_codes = a_codes;
    g.a_scales = a_scales;
    g.a_tscale = a_tscale;
    g.a_per_row = 1;
    return launch_grouped_gemm(g, 1, stream);
}

size_t nvfp4_grouped_gemm_w4a4_workspace(int64_t a_rows, int64_t K)
{
    return gemm_w4a4_workspace(a_rows, K, FP4_SCALE_PER_ROW);
}

fp4_status nvfp4_grouped_gemm_w4a4(const void *a, int64_t a_rows, int64_t K, int64_t lda,
                                   const int32_t *row_index, const int32_t *group_offs, int64_t groups,
                                   int64_t rows, const uint8_t *w_codes, const uint8_t *w_scales,
                                   const float *w_tscale, int64_t N, void *c, fp4_dtype ct, int64_t ldc, void *ws,
                                   size_t ws_bytes, hipStream_t stream)
{
    bool empty = false;
    FP4_TRY(check_grouped(a_rows, K, row_index, group_offs, groups, rows, N, 64, c, ct, ldc, &empty));
    if (empty) return FP4_OK;
    FP4_TRY(check_matrix(a, a_rows, K, lda, 2));
    if (a_rows * K > kMaxFlatElems) return FP4_ERR_SHAPE;
    FP4_TRY(check_grouped_limits(a_rows, K, lda, true, groups, rows, N));  // before A is quantized
    FP4_TRY(check_packed(w_codes, w_scales));
    if (!w_tscale) return FP4_ERR_NULL;
    if (!ws || !aligned16(ws) || ws_bytes < nvfp4_grouped_gemm_w4a4_workspace(a_rows, K))
        return FP4_ERR_WORKSPACE;
    FP4_TRY(check_device());
    size_t co, so, to;
    gemm_w4a4_workspace_offsets(a_rows, K, &co, &so, &to);
    uint8_t *base = reinterpret_cast<uint8_t *>(ws);
    float *at = reinterpret_cast<float *>(base + to);
    FP4_TRY(launch_nvfp4_quantize(a, FP4_BF16, a_rows, K, lda, base + co, base + so, at, FP4_SCALE_PER_ROW,
                                  nullptr, nullptr, stream));
    return nvfp4_grouped_gemm_w4a4_prequant(base + co, base + so, at, a_rows, K, row_index, group_offs, groups,
                                            rows, w_codes, w_scales, w_tscale, N, c, ct, ldc, stream);
}

}  // extern "C"

// -------------------------------------------- key-value cache, attention --

namespace {

int kv_bits(fp4_kv_format f) { return f == FP4_KV_BF16 ? 16 : f == FP4_KV_MXFP8 ? 8 : 4; }

int log2_of(int64_t v)
{
    int s = 0;
    while ((int64_t(1) << s) < v) ++s;
    return s;
}

fp4_status check_cache(const fp4_kv_cache *c)
{
    if (!c) return FP4_ERR_NULL;
    if (c->format < FP4_KV_BF16 || c->format > FP4_KV_MXFP4) return FP4_ERR_DTYPE;
    if (c->pages <= 0 || c->kv_heads <= 0 || c->kv_heads > 65535) return FP4_ERR_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return FP4_ERR_SHAPE;
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return FP4_ERR_SHAPE;
    if (c->pages >= k2GiB / c->page_size) return FP4_ERR_SHAPE;
    if (!c->k_codes || !c->v_codes) return FP4_ERR_NULL;
    if (!aligned16(c->k_codes) || !aligned16(c->v_codes)) return FP4_ERR_LAYOUT;
    if (c->format != FP4_KV_BF16) {
        if (!c->k_scales || !c->v_scales) return FP4_ERR_NULL;
        if (!aligned16(c->k_scales) || !aligned16(c->v_scales)) return FP4_ERR_LAYOUT;
    }
    if (c->format == FP4_KV_NVFP4 && (!c->k_tscale || !c->v_tscale)) return FP4_ERR_NULL;
    return FP4_OK;
}

// rows of head_dim elements of size es at any token / head strides that keep them
// 16-byte aligned; outputs also need rows that do not overlap (by these strides)
fp4_status check_heads(const void *p, int64_t tok, int64_t head, int64_t dim, size_t es, bool output)
{
    if (!p) return FP4_ERR_NULL;
    const int64_t least = output ? dim : 0;
    if (tok < least || head < least) return FP4_ERR_LAYOUT;
    if (!aligned16(p) || ((uint64_t)tok * es) % 16 != 0 || ((uint64_t)head * es) % 16 != 0) return FP4_ERR_LAYOUT;
    return FP4_OK;
}

fp4_status check_table(const int32_t *table, int64_t seqs, int64_t width, int64_t stride, const fp4_kv_cache *c)
{
    if (seqs <= 0 || seqs >= (1 << 24) || width <= 0 || width >= (int64_t(1) << 30) / c->page_size) return FP4_ERR_SHAPE;
    if (!table) return FP4_ERR_NULL;
    if (stride < width && seqs > 1) return FP4_ERR_LAYOUT;
    return FP4_OK;
}

// the prompt kernel addresses a tile of 64 keys with 32-bit offsets
constexpr int64_t kMaxTokenStride = int64_t(1) << 24;

bool valid_scale(float s) { return s >= 0.0f && s <= 1.0e30f; }

// Partial results of the decode kernel: two slots a workgroup
struct DecodeSpace {
    int part_heads;
    size_t ml_offset, bytes;
};

DecodeSpace decode_space(int64_t seqs, int64_t heads, const fp4_kv_cache *c, int64_t width)
{
    const int64_t group = heads / c->kv_heads;
    const int64_t grid = decode_grid(seqs, c->kv_heads, (group + 15) / 16, width * c->page_size);
    DecodeSpace s;
    s.part_heads = group < 16 ? (int)group : 16;
    s.ml_offset = (size_t)(2 * grid * s.part_heads * c->head_dim) * 4;
    s.bytes = align256(s.ml_offset + (size_t)(2 * grid * s.part_heads) * 8);
    return s;
}

KvArgs kv_args(const fp4_kv_cache *c)
{
    KvArgs a = {};
    a.codes[0] = reinterpret_cast<uint8_t *>(c->k_codes);
    a.codes[1] = reinterpret_cast<uint8_t *>(c->v_codes);
    a.scales[0] = c->k_scales;
    a.scales[1] = c->v_scales;
    a.tscale[0] = c->k_tscale;
    a.tscale[1] = c->v_tscale;
    a.kv_heads = (int)c->kv_heads;
    a.head_dim = (int)c->head_dim;
    a.page_shift = log2_of(c->page_size);
    a.pages = c->pages;
    return a;
}

// 8-value units of one call fit 32 bits
bool kv_units_ok(const fp4_kv_cache *c, int64_t tokens)
{
    return tokens < k2GiB && 2 * c->kv_heads * tokens < k2GiB / (c->head_dim / 8);
}

}  // namespace

extern "C" {

fp4_status kv_cache_append(const fp4_kv_cache *cache, const void *k, const void *v, fp4_dtype xt,
                           int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                           int64_t v_token_stride, int64_t v_head_stride, const int64_t *slots,
                           fp4_mx_rule rule, int32_t *nonfinite, hipStream_t stream)
{
    if (!valid_dtype(xt) || (rule != FP4_MX_OCP_FLOOR && rule != FP4_MX_CEIL)) return FP4_ERR_DTYPE;
    FP4_TRY(check_cache(cache));
    if (tokens < 0 || !kv_units_ok(cache, tokens)) return FP4_ERR_SHAPE;
    if (tokens == 0) return FP4_OK;
    FP4_TRY(check_heads(k, k_token_stride, k_head_stride, cache->head_dim, dsize(xt), false));
    FP4_TRY(check_heads(v, v_token_stride, v_head_stride, cache->head_dim, dsize(xt), false));
    if (!slots) return FP4_ERR_NULL;
    FP4_TRY(check_device());
    KvArgs a = kv_args(cache);
    a.tokens = tokens;
    a.x[0] = const_cast<void *>(k);
    a.x[1] = const_cast<void *>(v);
    a.tok[0] = k_token_stride;
    a.tok[1] = v_token_stride;
    a.head[0] = k_head_stride;
    a.head[1] = v_head_stride;
    a.slots = slots;
    a.rule = rule;
    a.nonfinite = nonfinite;
    return launch_kv_append(a, cache->format, xt, stream);
}

fp4_status kv_cache_read(const fp4_kv_cache *cache, const int32_t *block_table, int64_t seqs,
                         int64_t table_width, int64_t table_stride, const int32_t *cu_seqlens,
                         int64_t tokens, void *k, void *v, fp4_dtype yt, int64_t k_token_stride,
                         int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                         hipStream_t stream)
{
    if (!valid_dtype(yt)) return FP4_ERR_DTYPE;
    FP4_TRY(check_cache(cache));
    FP4_TRY(check_table(block_table, seqs, table_width, table_stride, cache));
    if (!cu_seqlens) return FP4_ERR_NULL;
    if (tokens < 0 || !kv_units_ok(cache, tokens)) return FP4_ERR_SHAPE;
    if (tokens == 0) return FP4_OK;
    FP4_TRY(check_heads(k, k_token_stride, k_head_stride, cache->head_dim, dsize(yt), true));
    FP4_TRY(check_heads(v, v_token_stride, v_head_stride, cache->head_dim, dsize(yt), true));
    FP4_TRY(check_device());
    KvArgs a = kv_args(cache);
    a.tokens = tokens;
    a.x[0] = k;
    a.x[1] = v;
    a.tok[0] = k_token_stride;
    a.tok[1] = v_token_stride;
    a.head[0] = k_head_stride;
    a.head[1] = v_head_stride;
    a.table = block_table;
    a.table_stride = table_stride;
    a.table_width = (int)table_width;
    a.seqs = (int)seqs;
    a.cu = cu_seqlens;
    return launch_kv_read(a, cache->format, yt, stream);
}

size_t attn_decode_paged_workspace(int64_t seqs, int64_t heads, const fp4_kv_cache *cache, int64_t table_width)
{
    if (!cache || seqs <= 0 || heads <= 0 || table_width <= 0 || cache->kv_heads <= 0 || cache->page_size <= 0 ||
        cache->head_dim <= 0 || heads % cache->kv_heads != 0)
        return 0;
    return decode_space(seqs, heads, cache, table_width).bytes;
}

fp4_status attn_decode_paged(const void *q, int64_t seqs, int64_t heads, int64_t q_seq_stride,
                             int64_t q_head_stride, const fp4_kv_cache *cache, const int32_t *block_table,
                             int64_t table_width, int64_t table_stride, const int32_t *seq_lens, float scale,
                             int64_t window, void *out, fp4_dtype ot, int64_t o_seq_stride,
                             int64_t o_head_stride, float *lse, void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (!valid_dtype(ot)) return FP4_ERR_DTYPE;
    FP4_TRY(check_cache(cache));
    FP4_TRY(check_table(block_table, seqs, table_width, table_stride, cache));
    if (heads <= 0 || heads > 65535 || heads % cache->kv_heads != 0 || window < 0 || !valid_scale(scale)) return FP4_ERR_SHAPE;
    const int64_t max_len = table_width * cache->page_size;
    const int64_t group = heads / cache->kv_heads, head_tiles = (group + 15) / 16;
    if (seqs * heads >= k2GiB || decode_units_bound(seqs, cache->kv_heads, head_tiles, max_len) >= k2GiB)
        return FP4_ERR_SHAPE;
    FP4_TRY(check_heads(q, q_seq_stride, q_head_stride, cache->head_dim, 2, false));
    FP4_TRY(check_heads(out, o_seq_stride, o_head_stride, cache->head_dim, dsize(ot), true));
    if (!seq_lens) return FP4_ERR_NULL;
    FP4_TRY(check_device());
    const DecodeSpace sp = decode_space(seqs, heads, cache, table_width);
    if (sp.bytes > 0 && (!ws || !aligned16(ws) || ws_bytes < sp.bytes)) return FP4_ERR_WORKSPACE;
    DecodeArgs a = {};
    a.q = reinterpret_cast<const uint16_t *>(q);
    a.q_seq = q_seq_stride;
    a.q_head = q_head_stride;
    a.k_codes = reinterpret_cast<const uint8_t *>(cache->k_codes);
    a.v_codes = reinterpret_cast<const uint8_t *>(cache->v_codes);
    a.k_scales = cache->k_scales;
    a.v_scales = cache->v_scales;
    a.k_tscale = cache->format == FP4_KV_NVFP4 ? cache->k_tscale : nullptr;
    a.v_tscale = cache->format == FP4_KV_NVFP4 ? cache->v_tscale : nullptr;
    a.table = block_table;
    a.table_stride = table_stride;
    a.seq_lens = seq_lens;
    a.seqs = (int)seqs;
    a.heads = (int)heads;
    a.kv_heads = (int)cache->kv_heads;
    a.group = (int)group;
    a.head_tiles = (int)head_tiles;
    a.head_dim = (int)cache->head_dim;
    a.page_shift = log2_of(cache->page_size);
    a.pages = (int)cache->pages;
    a.max_len = (int)max_len;
    a.scale_log2 = scale * 1.44269504f;
    a.window = window > max_len ? 0 : (int)window;
    a.out = out;
    a.out_bf16 = ot == FP4_BF16;
    a.o_seq = o_seq_stride;
    a.o_head = o_head_stride;
    a.lse = lse;
    a.part_o = reinterpret_cast<float *>(ws);
    a.part_ml = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(ws) + sp.ml_offset);
    a.part_heads = sp.part_heads;
    return launch_attn_decode(a, cache->format, stream);
}

size_t attn_prefill_workspace(int64_t q_tokens, int64_t heads, int64_t k_tokens, int64_t kv_heads, int64_t head_dim,
                              int64_t seqs)
{
    if (q_tokens <= 0 || heads <= 0 || kv_heads <= 0 || heads % kv_heads != 0 || head_dim <= 0 || seqs <= 0) return 0;
    const int64_t group = heads / kv_heads;
    const int splits = prefill_splits(q_tokens, k_tokens, seqs, kv_heads, group, head_dim, 0);  // (a window only lowers it)
    return align256(prefill_part_rows(q_tokens, seqs, kv_heads, group, splits) * (size_t)(head_dim + 2) * 4);
}

fp4_status attn_prefill(const void *q, int64_t q_tokens, int64_t heads, int64_t q_token_stride,
                        int64_t q_head_stride, const void *k, const void *v, int64_t k_tokens,
                        int64_t kv_heads, int64_t head_dim, int64_t k_token_stride, int64_t k_head_stride,
                        int64_t v_token_stride, int64_t v_head_stride, const int32_t *cu_q,
                        const int32_t *cu_k, int64_t seqs, float scale, int causal, int64_t window, void *out,
                        fp4_dtype ot, int64_t o_token_stride, int64_t o_head_stride, float *lse, void *ws,
                        size_t ws_bytes, hipStream_t stream)
{
    if (!valid_dtype(ot) || (causal != 0 && causal != 1)) return FP4_ERR_DTYPE;
    if (heads <= 0 || heads > 65535 || kv_heads <= 0 || heads % kv_heads != 0) return FP4_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return FP4_ERR_SHAPE;
    if (q_tokens < 0 || k_tokens < 0 || seqs <= 0 || seqs >= (1 << 24) || window < 0 || !valid_scale(scale)) return FP4_ERR_SHAPE;
    const int64_t group = heads / kv_heads;
    if (k_tokens >= k2GiB || q_tokens >= k2GiB / group) return FP4_ERR_SHAPE;
    if (prefill_grid(q_tokens, seqs, kv_heads, group) >= k2GiB) return FP4_ERR_SHAPE;
    if (!cu_q || !cu_k) return FP4_ERR_NULL;
    if (q_tokens == 0) return FP4_OK;
    FP4_TRY(check_heads(q, q_token_stride, q_head_stride, head_dim, 2, false));
    if (k_tokens > 0) {
        FP4_TRY(check_heads(k, k_token_stride, k_head_stride, head_dim, 2, false));
        FP4_TRY(check_heads(v, v_token_stride, v_head_stride, head_dim, 2, false));
        if (k_token_stride >= kMaxTokenStride || v_token_stride >= kMaxTokenStride) return FP4_ERR_LAYOUT;
    }
    FP4_TRY(check_heads(out, o_token_stride, o_head_stride, head_dim, dsize(ot), true));
    FP4_TRY(check_device());
    const size_t need = attn_prefill_workspace(q_tokens, heads, k_tokens, kv_heads, head_dim, seqs);
    if (need > 0 && (!ws || !aligned16(ws) || ws_bytes < need)) return FP4_ERR_WORKSPACE;
    PrefillArgs a = {};
    a.splits = prefill_splits(q_tokens, k_tokens, seqs, kv_heads, group, head_dim, window);
    a.part_o = reinterpret_cast<float *>(ws);
    a.part_ml = a.part_o + prefill_part_rows(q_tokens, seqs, kv_heads, group, a.splits) * head_dim;
    a.q = reinterpret_cast<const uint16_t *>(q);
    a.k = reinterpret_cast<const uint16_t *>(k);
    a.v = reinterpret_cast<const uint16_t *>(v);
    a.q_tok = q_token_stride;
    a.q_head = q_head_stride;
    a.k_tok = k_token_stride;
    a.k_head = k_head_stride;
    a.v_tok = v_token_stride;
    a.v_head = v_head_stride;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.seqs = (int)seqs;
    a.heads = (int)heads;
    a.kv_heads = (int)kv_heads;
    a.group = (int)group;
    a.head_dim = (int)head_dim;
    a.q_tokens = q_tokens;
    a.k_tokens = k_tokens;
    a.scale_log2 = scale * 1.44269504f;
    a.causal = causal;
    a.window = window >= k_tokens ? 0 : (int)window;
    a.out = out;
    a.out_bf16 = ot == FP4_BF16;
    a.o_tok = o_token_stride;
    a.o_head = o_head_stride;
    a.lse = lse;
    return launch_attn_prefill(a, stream);
}

}  // extern "C"

// ------------------------------------------- around the attention --

namespace {

struct Strides {
    int64_t tok, head;
};

// what qk_norm_rope and qk_norm_rope_append share: the numbers first, then the pointers
fp4_status check_norm(fp4_dtype xt, fp4_dtype yt, int64_t tokens, int64_t heads, int64_t kv_heads, int64_t dim, float eps,
                      int64_t rot, int interleaved)
{
    if (!valid_dtype(xt) || !valid_dtype(yt) || (interleaved != 0 && interleaved != 1)) return FP4_ERR_DTYPE;
    if (tokens < 0 || tokens >= k2GiB || heads <= 0 || heads > 65535 || kv_heads < 0 || kv_heads > 65535) return FP4_ERR_SHAPE;
    if (dim <= 0 || dim > 512 || dim % 8 != 0 || rot < 0 || rot > dim || rot % 16 != 0) return FP4_ERR_SHAPE;
    if (!(eps == 0.0f || (eps >= 1.0e-30f && eps <= 1.0e30f))) return FP4_ERR_SHAPE;
    return FP4_OK;
}

fp4_status check_weight(const float *w, int64_t stride)
{
    if (!w) return FP4_ERR_NULL;
    if (stride < 0 || stride % 4 != 0 || !aligned16(w)) return FP4_ERR_LAYOUT;
    return FP4_OK;
}

fp4_status check_angles(const int32_t *positions, const double *freqs, int64_t rot)
{
    if (rot == 0) return FP4_OK;
    if (!positions || !freqs) return FP4_ERR_NULL;
    return (reinterpret_cast<uintptr_t>(freqs) & 7u) == 0 ? FP4_OK : FP4_ERR_LAYOUT;
}

HeadNormArgs norm_args(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t dim, const float *qw, const float *kw,
                       int64_t qws, int64_t kws, float eps, const int32_t *positions, const double *freqs, int64_t rot,
                       int interleaved)
{
    HeadNormArgs a = {};
    a.w[0] = qw;
    a.w[1] = kw;
    a.w_head[0] = qws;
    a.w_head[1] = kws;
    a.positions = positions;
    a.freqs = freqs;
    a.tokens = tokens;
    a.heads = (int)heads;
    a.kv_heads = (int)kv_heads;
    a.dim = (int)dim;
    a.rot = (int)rot;
    a.interleaved = interleaved;
    a.norm = eps > 0.0f;
    a.eps = eps;
    a.inv_dim = 1.0f / (float)dim;
    return a;
}

void set_rows(HeadNormArgs &a, int i, const void *x, Strides s)
{
    a.x[i] = x;
    a.x_tok[i] = s.tok;
    a.x_head[i] = s.head;
}

void set_out(HeadNormArgs &a, int i, void *y, Strides s)
{
    a.y[i] = y;
    a.y_tok[i] = s.tok;
    a.y_head[i] = s.head;
}

fp4_status check_pool(const fp4_kv_pages *p)
{
    if (!p) return FP4_ERR_NULL;
    if (p->pages <= 0 || p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1))) return FP4_ERR_SHAPE;
    if (p->pages >= k2GiB / p->page_size) return FP4_ERR_SHAPE;
    if (!p->free_list || !p->state) return FP4_ERR_NULL;
    return FP4_OK;
}

fp4_status check_rows_of(const int32_t *table, int64_t seqs, int64_t width, int64_t stride, int64_t page_size)
{
    if (seqs <= 0 || seqs >= (1 << 24) || width <= 0 || width >= (int64_t(1) << 30) / page_size) return FP4_ERR_SHAPE;
    if (!table) return FP4_ERR_NULL;
    if (stride < width && seqs > 1) return FP4_ERR_LAYOUT;
    return FP4_OK;
}

PageArgs page_args(const fp4_kv_pages *p, int32_t *table, int64_t seqs, int64_t width, int64_t stride,
                   const int32_t *seq_lens, void *ws)
{
    PageArgs a = {};
    a.free_list = p->free_list;
    a.state_in = a.state_out = p->state;
    a.table = table;
    a.table_stride = stride;
    a.seq_lens = seq_lens;
    a.ws = reinterpret_cast<int32_t *>(ws);
    a.pages = (int)p->pages;
    a.page_shift = log2_of(p->page_size);
    a.width = (int)width;
    a.seqs = (int)seqs;
    return a;
}

// Workspace of beam_select: sums, then maxima, values and tokens of the parts
struct BeamSpace {
    int64_t parts;  // of all rows
    size_t top, value, token, bytes;
};

BeamSpace beam_space(int64_t batch, int64_t beams, int64_t vocab, int64_t k, fp4_dtype xt)
{
    BeamSpace s;
    s.parts = batch * beams * beam_shape(batch * beams, beams, vocab, k, xt).parts;
    s.top = align256((size_t)s.parts * 8);
    s.value = s.top + align256((size_t)s.parts * 4);
    s.token = s.value + align256((size_t)(s.parts * k) * 4);
    s.bytes = s.token + align256((size_t)(s.parts * k) * 4);
    return s;
}

// (a launch holds fewer than 2^32 threads: 64 for every 1024 logits of a row or part of them, at most 1024 for a group)
bool beam_sizes_ok(int64_t batch, int64_t beams, int64_t vocab, int64_t k)
{
    return batch > 0 && batch < (1 << 21) && beams > 0 && beams <= 64 && vocab > 0 && vocab <= (int64_t(1) << 30) / beams &&
           k > 0 && k <= 64 && k <= beams * vocab && batch * beams * ((vocab + 4095) / 4096) < (1 << 24);
}

}  // namespace

extern "C" {

fp4_status qk_norm_rope(const void *q, const void *k, fp4_dtype xt, int64_t tokens, int64_t heads, int64_t kv_heads,
                        int64_t head_dim, int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride,
                        int64_t k_head_stride, const float *q_weight, const float *k_weight,
                        int64_t q_weight_stride, int64_t k_weight_stride, float eps, const int32_t *positions,
                        const double *freqs, int64_t rot, int interleaved, void *q_out, void *k_out, fp4_dtype yt,
                        int64_t qo_token_stride, int64_t qo_head_stride, int64_t ko_token_stride,
                        int64_t ko_head_stride, hipStream_t stream)
{
    FP4_TRY(check_norm(xt, yt, tokens, heads, kv_heads, head_dim, eps, rot, interleaved));
    if (tokens == 0) return FP4_OK;
    FP4_TRY(check_heads(q, q_token_stride, q_head_stride, head_dim, dsize(xt), false));
    FP4_TRY(check_heads(q_out, qo_token_stride, qo_head_stride, head_dim, dsize(yt), true));
    if (eps > 0.0f) FP4_TRY(check_weight(q_weight, q_weight_stride));
    if (kv_heads > 0) {
        FP4_TRY(check_heads(k, k_token_stride, k_head_stride, head_dim, dsize(xt), false));
        FP4_TRY(check_heads(k_out, ko_token_stride, ko_head_stride, head_dim, dsize(yt), true));
        if (eps > 0.0f) FP4_TRY(check_weight(k_weight, k_weight_stride));
    }
    FP4_TRY(check_angles(positions, freqs, rot));
    FP4_TRY(check_device());
    HeadNormArgs a = norm_args(tokens, heads, kv_heads, head_dim, q_weight, k_weight, q_weight_stride, k_weight_stride, eps,
                               positions, freqs, rot, interleaved);
    set_rows(a, 0, q, {q_token_stride, q_head_stride});
    set_rows(a, 1, k, {k_token_stride, k_head_stride});
    set_out(a, 0, q_out, {qo_token_stride, qo_head_stride});
    set_out(a, 1, k_out, {ko_token_stride, ko_head_stride});
    return launch_head_norm_rope(a, -1, xt, yt, stream);
}

fp4_status qk_norm_rope_append(const fp4_kv_cache *cache, const void *q, const void *k, const void *v, fp4_dtype xt,
                               int64_t tokens, int64_t heads, int64_t q_token_stride, int64_t q_head_stride,
                               int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                               int64_t v_head_stride, const float *q_weight, const float *k_weight,
                               int64_t q_weight_stride, int64_t k_weight_stride, float eps,
                               const int32_t *positions, const double *freqs, int64_t rot, int interleaved,
                               const int64_t *slots, fp4_mx_rule rule, int32_t *nonfinite, void *q_out,
                               fp4_dtype yt, int64_t qo_token_stride, int64_t qo_head_stride, hipStream_t stream)
{
    if (rule != FP4_MX_OCP_FLOOR && rule != FP4_MX_CEIL) return FP4_ERR_DTYPE;
    FP4_TRY(check_cache(cache));
    const int64_t dim = cache->head_dim;
    FP4_TRY(check_norm(xt, yt, tokens, heads, cache->kv_heads, dim, eps, rot, interleaved));
    if (tokens == 0) return FP4_OK;
    FP4_TRY(check_heads(q, q_token_stride, q_head_stride, dim, dsize(xt), false));
    FP4_TRY(check_heads(k, k_token_stride, k_head_stride, dim, dsize(xt), false));
    FP4_TRY(check_heads(v, v_token_stride, v_head_stride, dim, dsize(xt), false));
    FP4_TRY(check_heads(q_out, qo_token_stride, qo_head_stride, dim, dsize(yt), true));
    if (eps > 0.0f) {
        FP4_TRY(check_weight(q_weight, q_weight_stride));
        FP4_TRY(check_weight(k_weight, k_weight_stride));
    }
    FP4_TRY(check_angles(positions, freqs, rot));
    if (!slots) return FP4_ERR_NULL;
    FP4_TRY(check_device());
    HeadNormArgs a = norm_args(tokens, heads, cache->kv_heads, dim, q_weight, k_weight, q_weight_stride, k_weight_stride, eps,
                               positions, freqs, rot, interleaved);
    set_rows(a, 0, q, {q_token_stride, q_head_stride});
    set_rows(a, 1, k, {k_token_stride, k_head_stride});
    set_rows(a, 2, v, {v_token_stride, v_head_stride});
    set_out(a, 0, q_out, {qo_token_stride, qo_head_stride});
    a.kv = kv_args(cache);
    a.kv.tokens = tokens;
    a.kv.slots = slots;
    a.kv.rule = rule;
    a.kv.nonfinite = nonfinite;
    return launch_head_norm_rope(a, cache->format, xt, yt, stream);
}

size_t kv_pages_extend_workspace(int64_t seqs, int64_t tokens)
{
    return seqs <= 0 || tokens < 0 ? 0 : pages_extend_bytes(seqs, tokens);
}

fp4_status kv_pages_extend(const fp4_kv_pages *pool, int32_t *block_table, int64_t seqs, int64_t table_width,
                           int64_t table_stride, const int32_t *seq_lens, const int32_t *new_lens, int64_t tokens,
                           int32_t *lens_out, int32_t *state_out, int64_t *slots, int32_t *positions,
                           int32_t *cu_q, int32_t *cu_k, void *ws, size_t ws_bytes, hipStream_t stream)
{
    FP4_TRY(check_pool(pool));
    FP4_TRY(check_rows_of(block_table, seqs, table_width, table_stride, pool->page_size));
    if (tokens < 0 || tokens >= (int64_t(1) << 30)) return FP4_ERR_SHAPE;
    if (!seq_lens || !new_lens || !lens_out || !state_out) return FP4_ERR_NULL;
    if (tokens > 0 && (!slots || !positions)) return FP4_ERR_NULL;
    const size_t need = pages_extend_bytes(seqs, tokens);
    if (need > 0 && (!ws || !aligned16(ws) || ws_bytes < need)) return FP4_ERR_WORKSPACE;
    FP4_TRY(check_device());
    PageArgs a = page_args(pool, block_table, seqs, table_width, table_stride, seq_lens, ws);
    a.new_lens = new_lens;
    a.lens_out = lens_out;
    a.state_out = state_out;
    a.slots = slots;
    a.positions = positions;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.tokens = tokens;
    return launch_pages_extend(a, stream);
}

size_t kv_pages_collect_workspace(int64_t pages, int64_t seqs, int64_t table_width)
{
    return pages <= 0 || seqs <= 0 || table_width <= 0 ? 0 : pages_collect_bytes(pages, seqs, table_width);
}

fp4_status kv_pages_collect(const fp4_kv_pages *pool, const int32_t *block_table, int64_t seqs, int64_t table_width,
                            int64_t table_stride, const int32_t *seq_lens, void *ws, size_t ws_bytes,
                            hipStream_t stream)
{
    FP4_TRY(check_pool(pool));
    FP4_TRY(check_rows_of(block_table, seqs, table_width, table_stride, pool->page_size));
    if (!seq_lens) return FP4_ERR_NULL;
    const size_t need = pages_collect_bytes(pool->pages, seqs, table_width);
    if (need > 0 && (!ws || !aligned16(ws) || ws_bytes < need)) return FP4_ERR_WORKSPACE;
    FP4_TRY(check_device());
    return launch_pages_collect(
        page_args(pool, const_cast<int32_t *>(block_table), seqs, table_width, table_stride, seq_lens, ws), stream);
}

fp4_status kv_pages_reorder(const int32_t *block_table, int64_t batch, int64_t beams, int64_t table_width,
                            int64_t table_stride, const int32_t *seq_lens, const int32_t *parents,
                            int64_t page_size, int32_t *out, int64_t out_stride, int32_t *copies,
                            hipStream_t stream)
{
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return FP4_ERR_SHAPE;
    if (batch <= 0 || batch >= (1 << 24) || beams <= 0 || beams > 64) return FP4_ERR_SHAPE;
    FP4_TRY(check_rows_of(block_table, batch * beams, table_width, table_stride, page_size));
    FP4_TRY(check_rows_of(out, batch * beams, table_width, out_stride, page_size));
    if (pages_reorder_grid(batch, table_width) >= (1 << 24)) return FP4_ERR_SHAPE;
    if (out == block_table && out_stride != table_stride) return FP4_ERR_LAYOUT;
    if (!seq_lens || !parents || !copies) return FP4_ERR_NULL;
    FP4_TRY(check_device());
    BeamTableArgs a = {};
    a.table = block_table;
    a.table_stride = table_stride;
    a.out = out;
    a.out_stride = out_stride;
    a.seq_lens = seq_lens;
    a.parents = parents;
    a.copies = copies;
    a.batch = (int)batch;
    a.beams = (int)beams;
    a.width = (int)table_width;
    a.page_shift = log2_of(page_size);
    return launch_pages_reorder(a, stream);
}

fp4_status kv_cache_copy(const fp4_kv_cache *cache, const int32_t *copies, int64_t n, hipStream_t stream)
{
    FP4_TRY(check_cache(cache));
    if (n < 0 || n >= (int64_t(1) << 23) / cache->kv_heads) return FP4_ERR_SHAPE;
    if (n == 0) return FP4_OK;
    if (!copies) return FP4_ERR_NULL;
    FP4_TRY(check_device());
    return launch_kv_copy(kv_args(cache), cache->format, copies, n, stream);
}

size_t beam_select_workspace(int64_t batch, int64_t beams, int64_t vocab, int64_t k, fp4_dtype xt)
{
    if (!valid_dtype(xt) || !beam_sizes_ok(batch, beams, vocab, k)) return 0;
    return beam_space(batch, beams, vocab, k, xt).bytes;
}

fp4_status beam_select(const void *logits, fp4_dtype xt, int64_t batch, int64_t beams, int64_t vocab, int64_t ld,
                       const float *scores, const uint8_t *done, int64_t end_token, int64_t k, float *out_scores,
                       int32_t *out_parents, int32_t *out_tokens, void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (!valid_dtype(xt)) return FP4_ERR_DTYPE;
    if (!beam_sizes_ok(batch, beams, vocab, k) || end_token < 0 || end_token >= vocab) return FP4_ERR_SHAPE;
    if (!logits || !scores || !out_scores || !out_parents || !out_tokens) return FP4_ERR_NULL;
    if (ld < vocab || (reinterpret_cast<uintptr_t>(logits) % dsize(xt)) != 0) return FP4_ERR_LAYOUT;
    const BeamSpace sp = beam_space(batch, beams, vocab, k, xt);
    if (!ws || !aligned16(ws) || ws_bytes < sp.bytes) return FP4_ERR_WORKSPACE;
    FP4_TRY(check_device());
    uint8_t *base = reinterpret_cast<uint8_t *>(ws);
    BeamArgs a = {};
    a.logits = logits;
    a.ld = ld;
    a.scores = scores;
    a.done = done;
    a.batch = (int)batch;
    a.beams = (int)beams;
    a.vocab = (int)vocab;
    a.k = (int)k;
    a.end_token = (int)end_token;
    a.part_sum = reinterpret_cast<double *>(base);
    a.part_top = reinterpret_cast<float *>(base + sp.top);
    a.part_value = reinterpret_cast<float *>(base + sp.value);
    a.part_token = reinterpret_cast<int32_t *>(base + sp.token);
    a.out_scores = out_scores;
    a.out_parents = out_parents;
    a.out_tokens = out_tokens;
    return launch_beam_select(a, xt, stream);
}

}  // extern "C"
