// head_norm.hip -- queries and keys between their projection and the attention: every head's row is
// normed (root mean square) and rotated by its token's position, in one pass; a second form writes
// the keys and the values into the paged cache in its format instead of giving key rows.
//
// For a row x of `dim` values, y = x (mean x^2 + eps)^-1/2 w; then each pair (y_i, y_j) of the first
// `rot` turns by the angle position * freqs[i]: (y_i c - y_j s, y_j c + y_i s), with j = i + rot/2 or,
// interleaved, neighbouring values.
//
// One lane holds 8 consecutive values, dim / 8 lanes (rounded up to a power of two) a row, so a wave
// holds up to 64 / that many rows at a time.  A wave takes one token and walks over its heads: the 8
// cosines and sines of a lane depend on the token and the lane's place in the row only, and are formed
// once a token, in place of a table that would have to be read.  Bound by memory where there are many tokens: 16384
// tokens of 40 + 8 heads of 128 in bf16, 403 MB, take 85 us (4.7 TB/s; a large copy runs at 5.2), one row a lane group
// at a time 128 us; 6001 tokens of 16 + 4 + 4 heads of 256 into a bf16 cache, 148 MB, 33 us.  By the launch where
// there are few: one token 3.8 us.
#include "quant_device.h"

namespace fp4k {

namespace {

// sin and cos of a quarter turns: position * freq is taken to quarter turns and reduced in 64 bits
// (2^31 positions at 1 radian each lose 2^-22 of a turn; in 32 bits a position of 10^6 would be off
// by 0.06 radian), the rest |t| <= 1/2 goes through polynomials of degree 9 and 8 fitted over that
// interval (largest error 9e-8).
__device__ __forceinline__ void turn(double position, double freq, float &c, float &s)
{
    const double a = position * (freq * 0.63661977236758134308);  // 2 / pi
    const double n = __builtin_rint(a);
    const float t = (float)(a - n), u = t * t;
    // the quarter, modulo 4: n - 4 rint(n / 4) is in [-2, 2] and exact
    const int q = (int)(float)__builtin_fma(-4.0, __builtin_rint(n * 0.25), n) & 3;
    float sn = __builtin_fmaf(u, 1.5820653061382473e-4f, -4.681266378611326e-3f);
    sn = __builtin_fmaf(u, sn, 0.07969257980585098f);
    sn = __builtin_fmaf(u, sn, -0.6459640860557556f);
    sn = __builtin_fmaf(u, sn, 1.5707963705062866f) * t;
    float cn = __builtin_fmaf(u, 9.0362987248227e-4f, -0.02086007036268711f);
    cn = __builtin_fmaf(u, cn, 0.25366920232772827f);
    cn = __builtin_fmaf(u, cn, -1.2337005138397217f);
    cn = __builtin_fmaf(u, cn, 1.0f);
    const float x = (q & 1) ? sn : cn, y = (q & 1) ? cn : sn;
    c = (q == 1 || q == 2) ? -x : x;
    s = (q & 2) ? -y : y;
}

// Sum over the 2^lane_shift neighbouring lanes of a row; every lane gets it, in the same order.
__device__ __forceinline__ float row_sum(float v, int lane_shift)
{
    if (lane_shift >= 1) v += xor1(v);
    if (lane_shift >= 2) v += xor2(v);
    if (lane_shift >= 3) v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, false));
    if (lane_shift >= 4) v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, false));
    if (lane_shift >= 5) v += __shfl_xor(v, 16, kWave);
    if (lane_shift >= 6) v += __shfl_xor(v, 32, kWave);
    return v;
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8])
{
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]),
                                                   bf16x2_rne(v[6], v[7]));
    } else {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// the place of a lane's 8 values among those of a cache's pages
__device__ __forceinline__ int64_t cache_unit(const KvArgs &a, int head, int64_t slot, uint32_t c8, int lane_shift)
{
    const int64_t page = slot >> a.page_shift;
    const uint32_t off = (uint32_t)slot & ((1u << a.page_shift) - 1u);
    return ((((page * a.kv_heads + head) << a.page_shift) + off) << lane_shift) + c8;
}

constexpr int kRowsOut = -1;  // FMT: key rows are outputs, there is no cache

// 8 values of a row into the cache (the lanes of a block come here together)
template <int FMT>
__device__ __forceinline__ void cache8(const KvArgs &a, int side, int head, int64_t slot, uint32_t c8, int lane_shift,
                                       const float (&v)[8])
{
    const int64_t page = slot >> a.page_shift;
    const uint32_t off = (uint32_t)slot & ((1u << a.page_shift) - 1u);
    const int64_t block = (page * a.kv_heads + head) << a.page_shift;
    uint8_t *codes = side ? a.codes[1] : a.codes[0], *scales = side ? a.scales[1] : a.scales[0];
    const int64_t unit = cache_unit(a, head, slot, c8, lane_shift);
    if constexpr (FMT == FP4_KV_BF16) {
        store8(reinterpret_cast<uint16_t *>(codes) + unit * 8, v);
    } else {
        constexpr int kBlkShift = FMT == FP4_KV_NVFP4 ? 1 : 2;  // lanes of a block
        constexpr int kUnitB = FMT == FP4_KV_MXFP8 ? 8 : 4;     // code bytes of a unit
        uint32_t byte;
        int bad = 0;
        const float s = FMT == FP4_KV_NVFP4 ? (side ? a.tscale[1] : a.tscale[0])[head] : 0.0f;
        const uint2 w = kv_encode8<FMT>(v, s, a.rule, byte, bad);
        uint8_t *cp = codes + unit * kUnitB;
        if constexpr (kUnitB == 8) *reinterpret_cast<uint2 *>(cp) = w;
        else *reinterpret_cast<uint32_t *>(cp) = w.x;
        if ((c8 & ((1u << kBlkShift) - 1u)) == 0u)
            scales[(block << (lane_shift - kBlkShift)) + ((c8 >> kBlkShift) << a.page_shift) + off] = (uint8_t)byte;
        if (bad && a.nonfinite) *a.nonfinite = 1;
    }
}

// 8 values to their place.  A bf16 cache takes the q rows' own store at another address: as two alternatives the compiler
// joined their ends into a store of 4 bytes and one of 12 (6001 tokens from memory 35.3 us, this way 33.2).
template <typename TO, int FMT>
__device__ __forceinline__ void put8(const HeadNormArgs &a, int side, int head, int64_t token, int64_t slot, bool stored, uint32_t c8,
                                     int lane_shift, const float (&v)[8])
{
    constexpr bool kSame = FMT == FP4_KV_BF16 && sizeof(TO) == 2;
    if (FMT == kRowsOut || kSame || side == 0) {
        const int64_t tok = FMT == kRowsOut && side ? a.y_tok[1] : a.y_tok[0], step = FMT == kRowsOut && side ? a.y_head[1] : a.y_head[0];
        TO *p = reinterpret_cast<TO *>(FMT == kRowsOut && side ? a.y[1] : a.y[0]) + token * tok + head * step + c8 * 8;
        if (kSame && side > 0) {
            if (!stored) return;
            p = reinterpret_cast<TO *>(side == 2 ? a.kv.codes[1] : a.kv.codes[0]) + cache_unit(a.kv, head, slot, c8, lane_shift) * 8;
        }
        store8(p, v);
    } else if constexpr (FMT != kRowsOut) {
        if (stored) cache8<FMT>(a.kv, side - 1, head, slot, c8, lane_shift, v);
    }
}

// How the two values of a pair meet: neighbours of a lane (interleaved), lanes 8 or 4 apart by DPP (half-split, rot
// 128 or 64), or any lanes by a shuffle.  (DPP / the shuffle for these too, us: in fp32 4096 tokens of 16 + 4 heads of 128
// 16.9 / 18.2, 8192 of 32 + 8 of 64 26.9 / 29.3; in bf16 16384 of 40 + 8 of 128 71.1 / 72.3, of 32 + 8 of 64 30.7 / 30.7;
// cache writes within 2% either way.)
enum { kPairLane = 0, kPair8 = 1, kPair4 = 2, kPairAny = 3 };

template <int PAIR>
__device__ __forceinline__ float partner_of(float v, int lane)
{
    if constexpr (PAIR == kPair8) return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x128, 0xF, 0xF, false));
    else if constexpr (PAIR == kPair4)  // lane ^ 7, then ^ 3
        return __int_as_float(__builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, false),
                                                       0x1B, 0xF, 0xF, false));
    else return __shfl(v, lane, kWave);
}

template <typename T>
struct Raw {  // 8 values as they are in memory
    uint4 w[sizeof(T) / 2];
    template <bool ONCE>
    __device__ __forceinline__ void load(const T *p)
    {
        const u32x4 *q = reinterpret_cast<const u32x4 *>(p);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            const u32x4 r = ONCE ? __builtin_nontemporal_load(q + i) : q[i];
            w[i] = make_uint4(r[0], r[1], r[2], r[3]);
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                v[i] = __uint_as_float((&w[0].x)[i]);
                v[4 + i] = __uint_as_float((&w[1].x)[i]);
            } else {
                v[2 * i] = __uint_as_float((&w[0].x)[i] << 16);
                v[2 * i + 1] = __uint_as_float((&w[0].x)[i] & 0xFFFF0000u);
            }
        }
    }
};

// A wave's passes go over the heads of q, then k, then v, each a multiple of the rows that a pass holds, so
// that the side of a pass is the same in all lanes.  The rows of U passes are requested together.
template <typename TI, typename TO, int FMT, int PAIR, bool ONCE>
__global__ __launch_bounds__(64) void k_head_norm_rope(HeadNormArgs a, int lane_shift)
{
    constexpr int U = 2;
    const int64_t token = a.first + (int64_t)blockIdx.x;
    const int lane = threadIdx.x, row = lane >> lane_shift;
    const uint32_t c8 = lane & ((1u << lane_shift) - 1u);
    const int e0 = (int)c8 * 8, once = 64 >> lane_shift;
    const int p0 = (int)blockIdx.y * a.slice_passes, p1 = min(a.passes[2], p0 + a.slice_passes);

    struct Pass {
        int side, head;
        bool here;
    };
    auto pass = [&](int p) {
        Pass x;
        x.side = p < a.passes[0] ? 0 : p < a.passes[1] ? 1 : 2;
        x.head = (p - (x.side == 0 ? 0 : x.side == 1 ? a.passes[0] : a.passes[1])) * once + row;
        x.here = e0 < a.dim && p < p1 && x.head < (x.side == 0 ? a.heads : a.kv_heads);
        return x;
    };
    auto request = [&](int p, Raw<TI> &raw) {
        const Pass x = pass(p);
        const TI *base = reinterpret_cast<const TI *>(x.side == 0 ? a.x[0] : x.side == 1 ? a.x[1] : a.x[2]);
        const int64_t tok = x.side == 0 ? a.x_tok[0] : x.side == 1 ? a.x_tok[1] : a.x_tok[2];
        const int64_t step = x.side == 0 ? a.x_head[0] : x.side == 1 ? a.x_head[1] : a.x_head[2];
#pragma unroll
        for (uint4 &w : raw.w) w = make_uint4(0, 0, 0, 0);
        if (x.here) raw.template load<ONCE>(base + token * tok + x.head * step + e0);
    };
    Raw<TI> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) request(p0 + u, raw[u]);

    // cosines and sines of this lane's values: the sign of the partner's share is in sn
    const bool turns = e0 < a.rot;
    const int half = a.rot >> 1;
    float cs[8], sn[8];
    int partner = lane;
    if (turns) {
        const double pos = (double)a.positions[token];
        if constexpr (PAIR == kPairLane) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float c, s;
                turn(pos, a.freqs[(e0 >> 1) + i], c, s);
                cs[2 * i] = cs[2 * i + 1] = c;
                sn[2 * i] = -s;
                sn[2 * i + 1] = s;
            }
        } else {
            const bool upper = e0 >= half;  // rot is a multiple of 16: a lane lies on one side
            partner = upper ? lane - (half >> 3) : lane + (half >> 3);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                turn(pos, a.freqs[e0 - (upper ? half : 0) + i], cs[i], sn[i]);
                if (!upper) sn[i] = -sn[i];
            }
        }
    }
    int64_t slot = -1;
    if constexpr (FMT != kRowsOut) slot = a.kv.slots[token];
    const bool stored = FMT != kRowsOut && slot >= 0 && slot < (a.kv.pages << a.kv.page_shift);

    bool left = false;  // a row of this lane is not done yet
    for (int p = p0; p < p1; p += U) {
        Raw<TI> next[U];
        if (p + U < p1) {
#pragma unroll
            for (int u = 0; u < U; ++u) request(p + U + u, next[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p + u >= p1) break;
            const Pass x = pass(p + u);
            bool here = x.here;
            float v[8];
            raw[u].get(v);
            if (x.side < 2) {
                if (a.norm) {
                    float ss = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(v[i], v[i], ss);
                    const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(row_sum(ss, lane_shift), a.inv_dim, a.eps));
                    float w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (x.here) Vec8<float>::load((x.side ? a.w[1] : a.w[0]) + x.head * (x.side ? a.w_head[1] : a.w_head[0]) + e0, w);
                    here &= inv != 0.0f;
                    left |= inv == 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = v[i] * inv * w[i];
                }
                if (a.rot > 0) {
                    float q[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) q[i] = PAIR == kPairLane ? v[i ^ 1] : partner_of<PAIR>(v[i], partner);
                    if (turns) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(v[i], cs[i], q[i] * sn[i]);
                    }
                }
            }
            if (!here) continue;
            put8<TO, FMT>(a, x.side, x.head, token, slot, stored, c8, lane_shift, v);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = next[u];
    }

    // Rows of values past 10^18, whose squares have no place in fp32 (the root's inverse is 0), were left as they are.  They are
    // taken 2^-70 times: 512 squares of any size have room then (2^125), and only bits below 2^-79 are lost, of a row whose root
    // mean square is above 2^59.  (A test within the loop, with this work behind it, kept its passes' chains from running beside
    // each other: one token 3.22 -> 3.5 us, 16384 70 -> 73.  This way 3.26 and 70.)
    if (!__ballot(left)) return;
    for (int p = p0; p < min(p1, a.passes[1]); ++p) {
        const Pass x = pass(p);
        request(p, raw[0]);
        float v[8], ss = 0.0f, w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        raw[0].get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(v[i], v[i], ss);
        const bool over = row_sum(ss, lane_shift) == __builtin_inff();
        ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] *= 0x1p-70f;
            ss = __builtin_fmaf(v[i], v[i], ss);
        }
        const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(row_sum(ss, lane_shift), a.inv_dim, a.eps * 0x1p-140f));
        if (x.here) Vec8<float>::load((x.side ? a.w[1] : a.w[0]) + x.head * (x.side ? a.w_head[1] : a.w_head[0]) + e0, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * inv * w[i];
        if (a.rot > 0) {
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = PAIR == kPairLane ? v[i ^ 1] : partner_of<PAIR>(v[i], partner);
            if (turns) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(v[i], cs[i], q[i] * sn[i]);
            }
        }
        if (!x.here || !over) continue;
        put8<TO, FMT>(a, x.side, x.head, token, slot, stored, c8, lane_shift, v);
    }
}

}  // namespace

template <typename TI, typename TO, int FMT, int PAIR>
static void launch_pair(HeadNormArgs a, int lane_shift, hipStream_t st)
{
    const int once = 64 >> lane_shift;
    a.passes[0] = (a.heads + once - 1) / once;
    a.passes[1] = a.passes[0] + (a.kv_heads + once - 1) / once;
    a.passes[2] = a.passes[1] + (FMT == kRowsOut ? 0 : (a.kv_heads + once - 1) / once);
    // A wave a token (the angles are formed once), or as many as give the chip 8 waves a SIMD, the most it holds (2 / 4 / 8 /
    // 16: 512 tokens of 40 + 8 heads of 128 6.3 / 6.1 / 6.8 / 6.9 us, 2048 17.2 / 13.9 / 13.5 / 14.3, 4096 22.4 / 22.4 / 19.7 /
    // 21.8).  Workgroups of one wave: four take the same time.
    int64_t slices = 32 * device_cu_count() / a.tokens;
    slices = slices < 1 ? 1 : slices > a.passes[2] ? a.passes[2] : slices;
    a.slice_passes = (int)((a.passes[2] + slices - 1) / slices);
    // Rows past the caches' size are read with the non-temporal hint: 403 MB in and out 84 us, 87 us without it
    // (74 and 87 when the outputs' memory is used again and again); between
    // a projection and the attention of its 8192 tokens (117 MB in) 1 to 2.5% of the whole chain's 640 us, at 16384 0.5%,
    // at 4096 (59 MB) and below none, while there rows that were used shortly before come back from the caches (4096
    // tokens read again and again: 25 us, 31 us with the hint).  Streaming stores are of no clear use there
    // (the chain at 4096 tokens 331 -> 335 us, at 8192 647 -> 643, at 16384 1233 -> 1235).
    const int64_t bytes = a.tokens * (a.heads + (FMT == kRowsOut ? 1 : 2) * a.kv_heads) * a.dim * (int64_t)sizeof(TI);
    const bool once_only = bytes >= (int64_t(96) << 20);
    // a launch holds fewer than 2^32 threads
    const int64_t slabs = (a.passes[2] + a.slice_passes - 1) / a.slice_passes, most = (int64_t(1) << 25) / slabs;
    for (a.first = 0; a.first < a.tokens; a.first += most) {
        const int64_t n = a.tokens - a.first < most ? a.tokens - a.first : most;
        const dim3 grid((unsigned)n, (unsigned)slabs);
        if (once_only) hipLaunchKernelGGL((k_head_norm_rope<TI, TO, FMT, PAIR, true>), grid, dim3(64), 0, st, a, lane_shift);
        else hipLaunchKernelGGL((k_head_norm_rope<TI, TO, FMT, PAIR, false>), grid, dim3(64), 0, st, a, lane_shift);
    }
}

template <typename TI, typename TO, int FMT>
static void launch_form(const HeadNormArgs &a, hipStream_t st)
{
    int lane_shift = 0;
    while ((8 << lane_shift) < a.dim) ++lane_shift;
    if (a.rot == 0 || a.interleaved) launch_pair<TI, TO, FMT, kPairLane>(a, lane_shift, st);
    else if (a.rot == 128) launch_pair<TI, TO, FMT, kPair8>(a, lane_shift, st);
    else if (a.rot == 64) launch_pair<TI, TO, FMT, kPair4>(a, lane_shift, st);
    else launch_pair<TI, TO, FMT, kPairAny>(a, lane_shift, st);
}

template <int FMT>
static void launch_types(const HeadNormArgs &a, fp4_dtype xt, fp4_dtype yt, hipStream_t st)
{
    if (xt == FP4_BF16) {
        if (yt == FP4_BF16) launch_form<uint16_t, uint16_t, FMT>(a, st);
        else launch_form<uint16_t, float, FMT>(a, st);
    } else {
        if (yt == FP4_BF16) launch_form<float, uint16_t, FMT>(a, st);
        else launch_form<float, float, FMT>(a, st);
    }
}

fp4_status launch_head_norm_rope(const HeadNormArgs &a, int fmt, fp4_dtype xt, fp4_dtype yt, hipStream_t st)
{
    if (fmt < 0) launch_types<kRowsOut>(a, xt, yt, st);
    else if (fmt == FP4_KV_BF16) launch_types<FP4_KV_BF16>(a, xt, yt, st);
    else if (fmt == FP4_KV_MXFP8) launch_types<FP4_KV_MXFP8>(a, xt, yt, st);
    else if (fmt == FP4_KV_NVFP4) launch_types<FP4_KV_NVFP4>(a, xt, yt, st);
    else launch_types<FP4_KV_MXFP4>(a, xt, yt, st);
    return hipGetLastError() == hipSuccess ? FP4_OK : FP4_ERR_HIP;
}

}  // namespace fp4k
