// quant_device.h -- the quantizers' device code: one lane, 8 consecutive values of a row.
//
// A 16-block is a lane pair, a 32-block a lane quad; block maxima are exchanged with DPP
// quad permutes, so the lanes of a block take every branch together.
#pragma once

#include "device_common.h"
#include "internal.h"

// IEEE round-to-nearest-even throughout: a contracted product and sum would round once
#pragma clang fp contract(off)

namespace fp4k {

template <typename T>
struct Vec8;

template <>
struct Vec8<float> {
    static __device__ __forceinline__ void load(const float *p, float v[8])
    {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        const float4 b = *reinterpret_cast<const float4 *>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

template <>
struct Vec8<uint16_t> {
    static __device__ __forceinline__ void load(const uint16_t *p, float v[8])
    {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};

__device__ __forceinline__ float amax8(const float v[8], int &bad)
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = __builtin_fabsf(v[i]);
        bad |= !__builtin_isfinite(a);
        m = fmaxf(m, a);
    }
    return m;
}

// Streaming (non-temporal) stores for the quantizers' outputs: each byte is written
// once and read, if at all, by a later kernel, so it need not stay in the caches.
// (The dequantizers keep ordinary stores: theirs cover 16 bytes of every 32 or 64
// per instruction, and as streaming stores those ran at half the rate.)
__device__ __forceinline__ void st_nt8(uint32_t v, uint8_t *p) { __builtin_nontemporal_store((uint8_t)v, p); }
__device__ __forceinline__ void st_nt32(uint32_t v, uint8_t *p)
{
    __builtin_nontemporal_store(v, reinterpret_cast<uint32_t *>(p));
}
__device__ __forceinline__ void st_nt64(uint32_t lo, uint32_t hi, uint8_t *p)
{
    __builtin_nontemporal_store(u32x2{lo, hi}, reinterpret_cast<u32x2 *>(p));
}

// ------------------------------------------- division by a shared divisor --
//
// Every value of a 16-block is divided by the same step d = fl32(E4M3(b) s), and
// every block byte of a row or tensor by the same 6 s.  gfx950's correctly
// rounded fp32 division (as the compiler emits it for a / b) is: pre-scale both
// operands (div_scale), y = rcp(b) refined by one Newton step, q0 = a y, then two
// remainder corrections q <- q + (a - b q) y by FMA, and a final special-value
// fix-up (div_fixup).  Only the product and the corrections depend on a, so
// rcp_refined() computes y once per divisor and div_refined() repeats the rest
// per value: a product and four FMAs in place of about eleven instructions.
// The pre-scaling is the identity (and the fix-up returns its input) when b and
// 1/b are normal, a is zero or not tiny (|a| >= 2^-103) and a / b is neither
// denormal nor within 2^96 of overflow.  nv_fast_scale(s) admits tensor scales
// s in [2^-50, 2^50]; every divisor is then in [2^-59, 2^59], and every quotient
// that can decide an E2M1 code or an E4M3 byte (a / b >= 2^-11) has a normal
// numerator, so it is formed exactly as by the division.  Smaller quotients
// land on code 0 / byte 0 either way.  Other scales take the IEEE division.

__device__ __forceinline__ bool nv_fast_scale(float s) { return s >= 0x1p-50f && s <= 0x1p50f; }

__device__ __forceinline__ float rcp_refined(float b)
{
    const float y0 = __builtin_amdgcn_rcpf(b);
    return __builtin_fmaf(__builtin_fmaf(-b, y0, 1.0f), y0, y0);
}

// Each correction is written q - (b q - a) y: the same value as q + (a - b q) y
// (round to nearest is symmetric, so the remainder is only negated), but a
// numerator of -0 then gives -0 (the sum -0 + -0), where the other order gives +0;
// so the quotient carries the sign of a in every case, as the division does.
__device__ __forceinline__ float div_refined(float a, float b, float y)
{
    const float q0 = a * y;
    const float q1 = __builtin_fmaf(-__builtin_fmaf(b, q0, -a), y, q0);
    return __builtin_fmaf(-__builtin_fmaf(b, q1, -a), y, q1);
}

// E4M3FN byte of one non-negative value (round to nearest even, saturating at 448).
__device__ __forceinline__ uint32_t e4m3_code_sat1(float q)
{
    typedef short v2i16 __attribute__((ext_vector_type(2)));
    const v2i16 r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v2i16{0, 0}, fminf(q, 448.0f), 0.0f, 1.0f, false);
    return (uint32_t)(uint16_t)r[0] & 0xFFu;
}

// The E4M3 block byte and the codes of one 8-element unit (lanes 2i, 2i + 1 hold
// one 16-block) on the fast path: bm8 = max|v| over the unit, y6 = rcp_refined(6 s).
// A block whose byte is 0 divides by s 2^20 instead of 0: its quotients are then
// below 2^-27 and every code is the sign alone, as the definition asks.
__device__ __forceinline__ uint32_t nvfp4_unit_fast(const float v[8], float bm8, float s, float six_s, float y6,
                                                    uint32_t &code_word)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const float bm = fmaxf(bm8, xor1(bm8));
    const uint32_t b = e4m3_code_sat1(div_refined(bm, six_s, y6));
    const f32x2 bv = __builtin_amdgcn_cvt_pk_f32_fp8((int)b, false);
    const float d = b ? bv[0] * s : s * 0x1p20f;
    const float y = rcp_refined(d);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = div_refined(v[i], d, y);
    code_word = e2m1x8_code(q);
    return b;
}

// Codes of 8 values under divisor d (d == 0: signed zeros), nibble i = value i.
__device__ __forceinline__ uint32_t nvfp4_codes8(const float v[8], float d)
{
    if (d == 0.0f) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= ((__float_as_uint(v[i]) >> 28) & 8u) << (4 * i);
        return w;
    }
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] / d;  // correctly rounded
    return e2m1x8_code(q);
}

// ------------------------------------------------- key-value cache rows --

// codes of 8 values and their block's scale byte, in the cache's format; the lanes of a
// block (two for NVFP4, four for the MX formats) are neighbours
template <int FMT>
__device__ __forceinline__ uint2 kv_encode8(const float (&v)[8], float s, int rule, uint32_t &byte, int &bad)
{
    if constexpr (FMT == FP4_KV_NVFP4) {
        uint32_t w;
        const float bm8 = amax8(v, bad);
        const float six_s = 6.0f * s;
        if (nv_fast_scale(s)) {
            byte = nvfp4_unit_fast(v, bm8, s, six_s, rcp_refined(six_s), w);
        } else {
            const float bm = fmaxf(bm8, xor1(bm8));
            byte = bm == 0.0f ? 0u : e4m3x4_code_sat(bm / six_s, 0.0f, 0.0f, 0.0f) & 0xFFu;
            w = nvfp4_codes8(v, e4m3_value(byte) * s);
        }
        return make_uint2(w, 0u);
    } else {
        constexpr int kTop = FMT == FP4_KV_MXFP8 ? 8 : 2;  // the element type's largest exponent
        float bm = amax8(v, bad);
        bm = fmaxf(bm, xor1(bm));
        bm = fmaxf(bm, xor2(bm));
        int k = 0;
        byte = 0;
        if (bm != 0.0f) {
            k = __builtin_amdgcn_frexp_expf(bm) - 1 - kTop;  // floor(log2 bm) - kTop, exact
            if (rule == 1 && __builtin_amdgcn_frexp_mantf(bm) > (FMT == FP4_KV_MXFP8 ? 0.875f : 0.75f)) ++k;
            k = k < -127 ? -127 : (k > 127 ? 127 : k);
            byte = (uint32_t)(k + 127);
        }
        if constexpr (FMT == FP4_KV_MXFP4) {
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = __builtin_amdgcn_ldexpf(v[i], -k);  // exact; a zero keeps its sign
            return make_uint2(e2m1x8_code(q), 0u);
        } else {
            float q[8];
            uint32_t lo = 0, hi = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                q[i] = __builtin_amdgcn_ldexpf(__builtin_fabsf(v[i]), -k);
                const uint32_t sign = __float_as_uint(v[i]) >> 31;
                (i < 4 ? lo : hi) |= sign << (8 * (i & 3) + 7);
            }
            return make_uint2(e4m3x4_code_sat(q[0], q[1], q[2], q[3]) | lo, e4m3x4_code_sat(q[4], q[5], q[6], q[7]) | hi);
        }
    }
}

__device__ __forceinline__ uint32_t bf16x2_rne(float lo, float hi)
{
    const bf16x2 v = {(__bf16)lo, (__bf16)hi};
    uint32_t r;
    __builtin_memcpy(&r, &v, 4);
    return r;
}

}  // namespace fp4k
