// attn_decode.hip -- attention of one new token per sequence over the paged,
// block-scaled key-value cache (include/fp4blk.h, fp4_kv_cache).
//
// For sequence b and query head h, with keys j in [max(0, len - window), len):
//   t_j = scale q.k_j,  o = sum_j exp(t_j - lse) v_j,  lse = log sum_j exp(t_j).
//
// Bound: every cached byte in range is read once, for 4 D flop a key and query
// head: a few flop a byte, so the kernel is bound by HBM as long as the widening
// of the codes stays off the critical path.  All query heads of a key head's group
// (up to 16) are therefore taken together, as the columns of one MFMA tile.
//
// One wave, 32 keys at a time (two sub-tiles of 16 keys):
//   S^T = K Q^T  16x16x32 MFMA, rows = keys, columns = heads: the lane (head
//                lane & 15, group g = lane >> 4) holds keys 4g .. 4g+3 of each sub-tile.
//   O^T += V^T P^T  the same lane must supply 8 keys of P for its head as the B
//                operand.  The order of the contracted keys is free, so slot (g, j)
//                is defined as key 4g + j (j < 4) or 16 + 4g + j - 4: exactly the
//                keys the lane already holds.  P never leaves its lane.
//                V^T rows: lane & 15 owns D/16 consecutive d of those 8 keys, read
//                straight from memory and transposed in registers (byte permutes of
//                the widened pairs), so V needs no LDS either.
// The running maximum is common to the four lane groups and moves only when a new
// score exceeds it by more than 2^8 (log2 units: 8), so the exchange between lanes
// and the rescaling are rare; P stays below 2^8, which neither its 16-bit form nor the
// fp32 sums mind.  P is rounded to 16 bits (bf16, or f16 for NVFP4) because the matrix
// core takes 16-bit operands; sums, maxima and outputs stay fp32 until the store.
//
// Widening: E2M1 / E4M3 times a power of two is exact in bf16 (MXFP4, MXFP8); E2M1
// times E4M3 is exact in f16, so NVFP4 runs on f16 operands: q is scaled by a power
// of two that puts its largest value in [2^14, 2^15), which loses nothing that is
// not below 2^-39 of that value.
//
// Work split: a unit is kTile keys of one (sequence, key head, 16-head tile); all
// units are numbered and the workgroups take equal, contiguous ranges, so ragged
// batches balance without the host knowing any length.  A range that covers only
// part of a row leaves an unnormalised partial result (max, sum, O) in the
// workspace, and k_attn_decode_join adds them up.
#include "device_common.h"
#include "internal.h"

namespace fp4k {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32 * kWaves;  // keys of one work unit
constexpr float kLazy = 8.0f;       // log2 headroom before the running maximum moves

constexpr int kv_bits(int fmt) { return fmt == FP4_KV_BF16 ? 16 : fmt == FP4_KV_MXFP8 ? 8 : 4; }
constexpr int kv_block(int fmt) { return fmt == FP4_KV_NVFP4 ? 16 : 32; }

// ------------------------------------------------------------ work split --

// First key a sequence's tiles start at (32-aligned) and the number of its tiles;
// an empty sequence has one (empty) tile, whose workgroup writes the zero row.
struct SeqSpan {
    int len, start, a0, tiles;
};

__device__ __forceinline__ SeqSpan seq_span(const DecodeArgs &a, int b)
{
    SeqSpan s;
    int n = a.seq_lens[b];
    n = n < 0 ? 0 : n;
    s.len = n > a.max_len ? a.max_len : n;
    s.start = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
    s.a0 = s.start & ~31;
    s.tiles = (s.len - s.a0 + kTile - 1) / kTile;
    s.tiles = s.tiles < 1 ? 1 : s.tiles;
    return s;
}

__device__ __forceinline__ int wave_inclusive_sum(int v)
{
    const int lane = threadIdx.x & 63;
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(v, off, kWave);
        if (lane >= off) v += o;
    }
    return v;
}

// Total tiles of all sequences (of one row each).
__device__ __forceinline__ int total_tiles(const DecodeArgs &a)
{
    const int lane = threadIdx.x & 63;
    int sum = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += 64) sum += b0 + lane < a.seqs ? seq_span(a, b0 + lane).tiles : 0;
    sum = wave_inclusive_sum(sum);
    return __builtin_amdgcn_readlane(sum, 63);
}

// The sequence that holds tile x of the concatenated sequences (0 <= x < total),
// and the number of tiles before it.
__device__ __forceinline__ void find_seq(const DecodeArgs &a, int x, int &b, int &before)
{
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int b0 = 0;; b0 += 64) {
        const int t = b0 + lane < a.seqs ? seq_span(a, b0 + lane).tiles : 0;
        const int inc = wave_inclusive_sum(t);
        const int sum = __builtin_amdgcn_readlane(inc, 63);
        if (x < base + sum || b0 + 64 >= a.seqs) {
            const uint64_t past = __ballot(base + inc <= x);  // sequences that end at or before x
            int i = __builtin_popcountll(past);
            i = i > 63 ? 63 : i;
            b = b0 + i;
            before = base + __builtin_amdgcn_readlane(inc - t, i);
            return;
        }
        base += sum;
    }
}

// Tiles before sequence b.
__device__ __forceinline__ int tiles_before(const DecodeArgs &a, int b)
{
    const int lane = threadIdx.x & 63;
    int sum = 0;
    for (int b0 = 0; b0 < b; b0 += 64) sum += b0 + lane < b ? seq_span(a, b0 + lane).tiles : 0;
    sum = wave_inclusive_sum(sum);
    return __builtin_amdgcn_readlane(sum, 63);
}

// Workgroup w of `grid` takes units [start(w), start(w + 1)): the first `extra` of
// them one unit more than the others.
struct Share {
    int each, extra;
};
__device__ __forceinline__ Share share_of(int units, int grid) { return {units / grid, units % grid}; }
__device__ __forceinline__ int share_start(const Share &s, int w) { return w * s.each + (w < s.extra ? w : s.extra); }
__device__ __forceinline__ int share_owner(const Share &s, int u)
{
    const int head = s.extra * (s.each + 1);
    return u < head ? u / (s.each + 1) : s.extra + (u - head) / s.each;  // each == 0 only when u < head
}

// ---------------------------------------------------------------- layout --

template <int FMT, int D>
struct Cfg {
    static constexpr int kBits = kv_bits(FMT);
    static constexpr bool kF16 = FMT == FP4_KV_NVFP4;
    static constexpr bool kScaled = FMT != FP4_KV_BF16;
    static constexpr int kBlk = kv_block(FMT);
    static constexpr int kRow = D * kBits / 8;  // bytes of a cached row
    // K: a lane's share of a row is D/4 values, in loads of at most 16 bytes; load i
    // of group g covers d = i * 4 KV + g * KV + [0, KV)
    static constexpr int kKB = D * kBits / 32 < 16 ? D * kBits / 32 : 16;
    static constexpr int kKV = kKB * 8 / kBits;
    static constexpr int kKL = D / 4 / kKV;
    static constexpr int kKW = kKL * kKB / 4;  // dwords
    // blocks of one K load (NVFP4: up to two), and all of a lane
    static constexpr int kKS = kScaled ? (kKV > kBlk ? kKV / kBlk : 1) : 0;
    // V: lane n = lane & 15 owns D/16 values of a row, in loads of at most 16 bytes;
    // load h covers d = h * 16 VV + n * VV + [0, VV), within one scale block
    static constexpr int kVB = D * kBits / 128 < 16 ? D * kBits / 128 : 16;
    static constexpr int kVV = kVB * 8 / kBits;
    static constexpr int kVL = D / 16 / kVV;
    static constexpr int kVW = (kVB + 3) / 4;  // dwords of a load
    static constexpr int kSteps = D / 32;      // MFMA steps of S
    static constexpr int kDT = D / 16;         // MFMA tiles of O
};

template <int BYTES>
__device__ __forceinline__ void load_dwords(const uint8_t *p, uint32_t *w)
{
    if constexpr (BYTES == 2) w[0] = *reinterpret_cast<const uint16_t *>(p);
    else if constexpr (BYTES == 4) w[0] = *reinterpret_cast<const uint32_t *>(p);
    else if constexpr (BYTES == 8) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
        static_assert(BYTES == 16, "load width");
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    }
}

// The raw bytes of 32 keys and values, as they come from memory.
template <int FMT, int D>
struct Raw {
    using C = Cfg<FMT, D>;
    uint32_t k[2][C::kKW];
    uint32_t ks[2][C::kScaled ? C::kKL * C::kKS : 1];
    uint32_t v[8][C::kVL][C::kVW];
    uint32_t vs[2][C::kVL];  // scale bytes of keys 4g .. 4g+3 of each sub-tile
};

// 8 values -> the 16-bit MFMA fragment (4 dwords)
template <int FMT>
__device__ __forceinline__ uint4 widen8(const uint32_t *w, uint32_t scale_byte)
{
    uint4 r;
    if constexpr (FMT == FP4_KV_BF16) {
        r = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (FMT == FP4_KV_MXFP8) {
        const float s = __uint_as_float(scale_byte << 23);
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], s, false);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], s, true);
        const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], s, false);
        const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], s, true);
        __builtin_memcpy(&r.x, &a, 4);
        __builtin_memcpy(&r.y, &b, 4);
        __builtin_memcpy(&r.z, &c, 4);
        __builtin_memcpy(&r.w, &d, 4);
    } else if constexpr (FMT == FP4_KV_MXFP4) {
        const bf16x8 v = e2m1x8_bf16_pow2(w[0], __uint_as_float(scale_byte << 23));
        __builtin_memcpy(&r, &v, 16);
    } else {
        const f16x2 e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scale_byte, 1.0f, false);
        const f16x2 s = {e[0], e[0]};
        const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[0], 1.0f, 0) * s;
        const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[0], 1.0f, 1) * s;
        const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[0], 1.0f, 2) * s;
        const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[0], 1.0f, 3) * s;
        __builtin_memcpy(&r.x, &a, 4);
        __builtin_memcpy(&r.y, &b, 4);
        __builtin_memcpy(&r.z, &c, 4);
        __builtin_memcpy(&r.w, &d, 4);
    }
    return r;
}

// The widened pair (values 2p, 2p + 1) of a load's bytes.
template <int FMT>
__device__ __forceinline__ uint32_t widen_pair(const uint32_t *w, int p, uint32_t scale_byte)
{
    uint32_t r;
    if constexpr (FMT == FP4_KV_BF16) {
        r = w[p];
    } else if constexpr (FMT == FP4_KV_MXFP8) {
        const float s = __uint_as_float(scale_byte << 23);
        const bf16x2 a = (p & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[p >> 1], s, true)
                                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[p >> 1], s, false);
        __builtin_memcpy(&r, &a, 4);
    } else if constexpr (FMT == FP4_KV_MXFP4) {
        const float s = __uint_as_float(scale_byte << 23);
        const uint32_t x = w[p >> 2];
        const bf16x2 a = (p & 3) == 0   ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, s, 0)
                         : (p & 3) == 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, s, 1)
                         : (p & 3) == 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, s, 2)
                                        : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, s, 3);
        __builtin_memcpy(&r, &a, 4);
    } else {
        const f16x2 e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scale_byte, 1.0f, false);
        const f16x2 s = {e[0], e[0]};
        const uint32_t x = w[p >> 2];
        const f16x2 a = (p & 3) == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(x, 1.0f, 0)
                        : (p & 3) == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(x, 1.0f, 1)
                        : (p & 3) == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(x, 1.0f, 2)
                                       : __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(x, 1.0f, 3);
        const f16x2 m = a * s;
        __builtin_memcpy(&r, &m, 4);
    }
    return r;
}

template <bool F16>
__device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c)
{
    if constexpr (F16) {
        f16x8 x, y;
        __builtin_memcpy(&x, &a, 16);
        __builtin_memcpy(&y, &b, 16);
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
    }
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if constexpr (F16) {
        const f16x2 v = {(_Float16)lo, (_Float16)hi};
        __builtin_memcpy(&r, &v, 4);
    } else {
        const bf16x2 v = {(__bf16)lo, (__bf16)hi};
        __builtin_memcpy(&r, &v, 4);
    }
    return r;
}

__device__ __forceinline__ float xor16_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16, kWave));
    return fmaxf(v, __shfl_xor(v, 32, kWave));
}
__device__ __forceinline__ float xor16_sum(float v)
{
    v += __shfl_xor(v, 16, kWave);
    return v + __shfl_xor(v, 32, kWave);
}

}  // namespace

template <int FMT, int D>
__global__ __launch_bounds__(256) void k_attn_decode(DecodeArgs a)
{
    using C = Cfg<FMT, D>;
    using R = Raw<FMT, D>;
    __shared__ f32x4 sm_o[2][C::kDT][64];
    __shared__ float sm_m[kWaves][16], sm_l[kWaves][16];
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    const int rows = a.kv_heads * a.head_tiles;
    const int units = total_tiles(a) * rows;
    const int grid = (int)gridDim.x < units ? (int)gridDim.x : units;
    const int wg = blockIdx.x;
    if (wg >= grid) return;
    const Share sh = share_of(units, grid);
    const int u_begin = share_start(sh, wg), u_end = share_start(sh, wg + 1);

    int b, before;
    find_seq(a, u_begin / rows, b, before);
    SeqSpan sp = seq_span(a, b);
    int base = before * rows;  // first unit of sequence b
    int slot = 2 * wg;
    for (int u = u_begin; u < u_end;) {
        while (u >= base + sp.tiles * rows) {
            base += sp.tiles * rows;
            sp = seq_span(a, ++b);
        }
        const int r = (u - base) / sp.tiles;
        const int t0 = (u - base) - r * sp.tiles;
        int t1 = t0 + (u_end - u);
        t1 = t1 > sp.tiles ? sp.tiles : t1;
        const int hkv = r / a.head_tiles, h0 = (r - hkv * a.head_tiles) * 16;
        const int nh = a.group - h0 < 16 ? a.group - h0 : 16;  // query heads of this tile
        const int head0 = hkv * a.group + h0;

        // ---- q: the B operand, lane n = head, the same order of d as K's loads
        uint4 q[C::kSteps];
        float c = a.scale_log2;
        {
            const uint16_t *qp = a.q + b * a.q_seq + (int64_t)(head0 + n) * a.q_head;
#pragma unroll
            for (int s = 0; s < C::kSteps; ++s) {
                const int i = 8 * s / C::kKV, e = 8 * s % C::kKV;
                q[s] = make_uint4(0, 0, 0, 0);
                if (n < nh) q[s] = *reinterpret_cast<const uint4 *>(qp + i * 4 * C::kKV + g * C::kKV + e);
            }
            if constexpr (C::kF16) {
                float m = 0.0f;
#pragma unroll
                for (int s = 0; s < C::kSteps; ++s) {
                    const uint32_t w[4] = {q[s].x, q[s].y, q[s].z, q[s].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        m = fmaxf(m, fmaxf(__builtin_fabsf(__uint_as_float(w[i] << 16)),
                                           __builtin_fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
                }
                m = xor16_max(m);
                const int e = m > 0.0f && m < INFINITY ? 15 - __builtin_amdgcn_frexp_expf(m) : 0;
#pragma unroll
                for (int s = 0; s < C::kSteps; ++s) {
                    uint32_t w[4] = {q[s].x, q[s].y, q[s].z, q[s].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = pack2<true>(__builtin_amdgcn_ldexpf(__uint_as_float(w[i] << 16), e),
                                           __builtin_amdgcn_ldexpf(__uint_as_float(w[i] & 0xFFFF0000u), e));
                    q[s] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                c = __builtin_amdgcn_ldexpf(c * a.k_tscale[hkv], -e);
            }
        }

        f32x4 o[C::kDT];
#pragma unroll
        for (int i = 0; i < C::kDT; ++i) o[i] = f32x4{0, 0, 0, 0};
        float m = -INFINITY, l = 0.0f;

        const int32_t *table = a.table + b * a.table_stride;
        const int page_mask = (1 << a.page_shift) - 1;
        auto load = [&](int key0, R &x) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int s = key0 + 16 * j;
                const int last = s < sp.len ? s : sp.len - 1;  // a sub-tile past the end reads the last page
                int id = table[last >> a.page_shift];
                id = id < 0 ? 0 : (id >= a.pages ? a.pages - 1 : id);
                const int off = s & page_mask;
                const int64_t block = ((int64_t)id * a.kv_heads + hkv) << a.page_shift;
                const uint8_t *kp = a.k_codes + (block + off) * C::kRow + n * C::kRow + g * C::kKB;
#pragma unroll
                for (int i = 0; i < C::kKL; ++i) load_dwords<C::kKB>(kp + i * 4 * C::kKB, &x.k[j][i * (C::kKB / 4)]);
                const uint8_t *vp = a.v_codes + (block + off + 4 * g) * C::kRow + n * C::kVB;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int h = 0; h < C::kVL; ++h) load_dwords<C::kVB>(vp + t * C::kRow + h * 16 * C::kVB, x.v[4 * j + t][h]);
                if constexpr (C::kScaled) {
                    constexpr int kBlocks = D / C::kBlk;
                    const uint8_t *ksp = a.k_scales + block * kBlocks + off + n;
#pragma unroll
                    for (int i = 0; i < C::kKL; ++i)
#pragma unroll
                        for (int e = 0; e < C::kKS; ++e) {
                            const int blk = (i * 4 * C::kKV + g * C::kKV) / C::kBlk + e;
                            x.ks[j][i * C::kKS + e] = ksp[blk << a.page_shift];
                        }
                    const uint8_t *vsp = a.v_scales + block * kBlocks + off + 4 * g;
#pragma unroll
                    for (int h = 0; h < C::kVL; ++h) {
                        const int blk = (h * 16 * C::kVV + n * C::kVV) / C::kBlk;
                        x.vs[j][h] = *reinterpret_cast<const uint32_t *>(vsp + (blk << a.page_shift));
                    }
                }
            }
        };
        auto compute = [&](int key0, R &x) {
            f32x4 s[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                s[j] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int st = 0; st < C::kSteps; ++st) {
                    const int i = 8 * st / C::kKV, e = 8 * st % C::kKV;
                    const uint32_t sc = C::kScaled ? x.ks[j][i * C::kKS + e / C::kBlk] : 0;
                    s[j] = mfma16<C::kF16>(widen8<FMT>(&x.k[j][8 * st * C::kBits / 32], sc), q[st], s[j]);
                }
            }
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = s[i >> 2][i & 3] * c;
            if (key0 < sp.start || key0 + 32 > sp.len) {
                // keys out of range: no score, and their values (which may be anything) become 0
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int key = key0 + 16 * (i >> 2) + 4 * g + (i & 3);
                    const bool in = key >= sp.start && key < sp.len;
                    t[i] = in ? t[i] : -INFINITY;
#pragma unroll
                    for (int h = 0; h < C::kVL; ++h) {
#pragma unroll
                        for (int w = 0; w < C::kVW; ++w) x.v[i][h][w] = in ? x.v[i][h][w] : 0u;
                        if constexpr (C::kScaled)
                            x.vs[i >> 2][h] = in ? x.vs[i >> 2][h] : x.vs[i >> 2][h] & ~(0xFFu << (8 * (i & 3)));
                    }
                }
            }
            const float tm = fmaxf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), fmaxf(fmaxf(t[4], t[5]), fmaxf(t[6], t[7])));
            if (__ballot(tm > m + kLazy)) {
                const float mn = fmaxf(m, xor16_max(tm));
                const float alpha = mn == m ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
                m = mn;
                l *= alpha;
#pragma unroll
                for (int i = 0; i < C::kDT; ++i) o[i] *= alpha;
            }
            const float mm = m == -INFINITY ? 0.0f : m;
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = __builtin_amdgcn_exp2f(t[i] - mm);
                l += p[i];
            }
            const uint4 pf = make_uint4(pack2<C::kF16>(p[0], p[1]), pack2<C::kF16>(p[2], p[3]), pack2<C::kF16>(p[4], p[5]),
                                        pack2<C::kF16>(p[6], p[7]));
            // O^T: a pair of d at a time, its two rows of V^T gathered from the 8 keys
#pragma unroll
            for (int h = 0; h < C::kVL; ++h)
#pragma unroll
                for (int pr = 0; pr < C::kVV / 2; ++pr) {
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        w[i] = widen_pair<FMT>(x.v[i][h], pr, C::kScaled ? (x.vs[i >> 2][h] >> (8 * (i & 3))) & 0xFFu : 0u);
                    uint4 lo, hi;
                    lo.x = __builtin_amdgcn_perm(w[1], w[0], 0x05040100u);
                    lo.y = __builtin_amdgcn_perm(w[3], w[2], 0x05040100u);
                    lo.z = __builtin_amdgcn_perm(w[5], w[4], 0x05040100u);
                    lo.w = __builtin_amdgcn_perm(w[7], w[6], 0x05040100u);
                    hi.x = __builtin_amdgcn_perm(w[1], w[0], 0x07060302u);
                    hi.y = __builtin_amdgcn_perm(w[3], w[2], 0x07060302u);
                    hi.z = __builtin_amdgcn_perm(w[5], w[4], 0x07060302u);
                    hi.w = __builtin_amdgcn_perm(w[7], w[6], 0x07060302u);
                    const int i0 = h * C::kVV + 2 * pr;
                    o[i0] = mfma16<C::kF16>(lo, pf, o[i0]);
                    o[i0 + 1] = mfma16<C::kF16>(hi, pf, o[i0 + 1]);
                }
        };
        for (int t = t0; t < t1; ++t) {
            const int key0 = sp.a0 + t * kTile + wave * 32;
            if (key0 >= sp.len) break;
            R x;
            load(key0, x);
            compute(key0, x);
        }

        // ---- the four waves' results become one
        l = xor16_sum(l);
        if (lane < 16) {
            sm_m[wave][n] = m;
            sm_l[wave][n] = l;
        }
        __syncthreads();
        const float M = fmaxf(fmaxf(sm_m[0][n], sm_m[1][n]), fmaxf(sm_m[2][n], sm_m[3][n]));
        const float Ms = M == -INFINITY ? 0.0f : M;
        float L = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) L += sm_l[w][n] * __builtin_amdgcn_exp2f(sm_m[w][n] - Ms);
        const float beta = __builtin_amdgcn_exp2f(m - Ms);
#pragma unroll
        for (int i = 0; i < C::kDT; ++i) o[i] *= beta;
        if (wave >= 2)
#pragma unroll
            for (int i = 0; i < C::kDT; ++i) sm_o[wave - 2][i][lane] = o[i];
        __syncthreads();
        if (wave < 2)
#pragma unroll
            for (int i = 0; i < C::kDT; ++i) o[i] += sm_o[wave][i][lane];
        __syncthreads();
        if (wave == 1)
#pragma unroll
            for (int i = 0; i < C::kDT; ++i) sm_o[0][i][lane] = o[i];
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int i = 0; i < C::kDT; ++i) o[i] += sm_o[0][i][lane];
            if (n < nh) {
                const bool whole = t0 == 0 && t1 == sp.tiles;
                float *po = nullptr;
                float f = 1.0f;
                if (whole) {
                    f = L > 0.0f || L != L ? 1.0f / L : 0.0f;
                    if constexpr (C::kF16) f = L == 0.0f ? 0.0f : f * a.v_tscale[hkv];
                    if (a.lse && g == 0) a.lse[(int64_t)b * a.heads + head0 + n] = (M + __builtin_amdgcn_logf(L)) * 0.69314718f;
                } else {
                    po = a.part_o + ((int64_t)slot * a.part_heads + n) * D;
                    if (g == 0) {
                        a.part_ml[((int64_t)slot * a.part_heads + n) * 2] = M;
                        a.part_ml[((int64_t)slot * a.part_heads + n) * 2 + 1] = L;
                    }
                }
#pragma unroll
                for (int h = 0; h < C::kVL; ++h)
#pragma unroll
                    for (int rr = 0; rr < 4; ++rr) {
                        const int d = h * 16 * C::kVV + (4 * g + rr) * C::kVV;
#pragma unroll
                        for (int i = 0; i < C::kVV; i += 4) {
                            const int k = h * C::kVV + i;
                            const float4 v = make_float4(o[k][rr] * f, o[k + 1][rr] * f, o[k + 2][rr] * f, o[k + 3][rr] * f);
                            if (!whole) {
                                *reinterpret_cast<float4 *>(po + d + i) = v;
                            } else if (a.out_bf16) {
                                uint16_t *p = reinterpret_cast<uint16_t *>(a.out) + b * a.o_seq + (head0 + n) * a.o_head + d + i;
                                *reinterpret_cast<uint2 *>(p) = make_uint2(pack2<false>(v.x, v.y), pack2<false>(v.z, v.w));
                            } else {
                                float *p = reinterpret_cast<float *>(a.out) + b * a.o_seq + (head0 + n) * a.o_head + d + i;
                                *reinterpret_cast<float4 *>(p) = v;
                            }
                        }
                    }
            }
        }
        __syncthreads();
        u += t1 - t0;
        slot = 2 * wg + 1;
    }
}

// One workgroup per (sequence, query head): adds up the partial results of a row
// that several workgroups of k_attn_decode share.
template <int D>
__global__ __launch_bounds__(256) void k_attn_decode_join(DecodeArgs a, int grid_full)
{
    constexpr int kParts = 256 / D;
    __shared__ float sm[kParts][D];
    __shared__ float sm_l[kParts];
    const int b = blockIdx.x / a.heads, head = blockIdx.x - b * a.heads;
    const int hkv = head / a.group, hg = head - hkv * a.group, n = hg & 15;
    const int rows = a.kv_heads * a.head_tiles;
    const int units = total_tiles(a) * rows;
    const int grid = grid_full < units ? grid_full : units;
    const Share sh = share_of(units, grid);
    const int tiles = seq_span(a, b).tiles;
    const int r = hkv * a.head_tiles + (hg >> 4);
    const int u0 = tiles_before(a, b) * rows + r * tiles;
    const int w0 = share_owner(sh, u0), w1 = share_owner(sh, u0 + tiles - 1);
    if (w0 == w1) return;
    const int first = share_start(sh, w0) >= u0 ? 2 * w0 : 2 * w0 + 1;
    auto at = [&](int w) -> int64_t { return (int64_t)(w == w0 ? first : 2 * w) * a.part_heads + n; };
    float M = -INFINITY;
    for (int w = w0 + (threadIdx.x & 63); w <= w1; w += 64) M = fmaxf(M, a.part_ml[at(w) * 2]);
    M = wave_max(M);
    const float Ms = M == -INFINITY ? 0.0f : M;
    const int d = threadIdx.x % D, part = threadIdx.x / D;
    float acc = 0.0f, L = 0.0f;
    for (int w = w0 + part; w <= w1; w += kParts) {
        const int64_t i = at(w);
        const float f = __builtin_amdgcn_exp2f(a.part_ml[i * 2] - Ms);
        L += f * a.part_ml[i * 2 + 1];
        acc += f * a.part_o[i * D + d];
    }
    sm[part][d] = acc;
    if (d == 0) sm_l[part] = L;
    __syncthreads();
    if (part != 0) return;
    acc = 0.0f;
    L = 0.0f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        acc += sm[i][d];
        L += sm_l[i];
    }
    float f = L == 0.0f ? 0.0f : 1.0f / L;
    if (a.v_tscale) f *= a.v_tscale[hkv];
    acc *= f;
    const int64_t p = b * a.o_seq + head * a.o_head + d;
    if (a.out_bf16) reinterpret_cast<__bf16 *>(a.out)[p] = (__bf16)acc;
    else reinterpret_cast<float *>(a.out)[p] = acc;
    if (a.lse && d == 0) a.lse[(int64_t)b * a.heads + head] = (M + __builtin_amdgcn_logf(L)) * 0.69314718f;
}

int decode_grid(int64_t seqs, int64_t kv_heads, int64_t head_tiles, int64_t max_len)
{
    const int64_t units = seqs * kv_heads * head_tiles * ((max_len + 31 + kTile - 1) / kTile);
    const int64_t most = 4 * (int64_t)device_cu_count();
    return (int)(units < most ? units : most);
}

int64_t decode_units_bound(int64_t seqs, int64_t kv_heads, int64_t head_tiles, int64_t max_len)
{
    return seqs * kv_heads * head_tiles * ((max_len + 31 + kTile - 1) / kTile);
}

template <int FMT>
static void launch_fmt(const DecodeArgs &a, int grid, hipStream_t st)
{
    if (a.head_dim == 64) hipLaunchKernelGGL((k_attn_decode<FMT, 64>), dim3(grid), dim3(256), 0, st, a);
    else if (a.head_dim == 128) hipLaunchKernelGGL((k_attn_decode<FMT, 128>), dim3(grid), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_attn_decode<FMT, 256>), dim3(grid), dim3(256), 0, st, a);
}

fp4_status launch_attn_decode(const DecodeArgs &a, fp4_kv_format fmt, hipStream_t st)
{
    const int grid = decode_grid(a.seqs, a.kv_heads, a.head_tiles, a.max_len);
    if (fmt == FP4_KV_BF16) launch_fmt<FP4_KV_BF16>(a, grid, st);
    else if (fmt == FP4_KV_MXFP8) launch_fmt<FP4_KV_MXFP8>(a, grid, st);
    else if (fmt == FP4_KV_NVFP4) launch_fmt<FP4_KV_NVFP4>(a, grid, st);
    else launch_fmt<FP4_KV_MXFP4>(a, grid, st);
    const dim3 jg((unsigned)(a.seqs * a.heads));
    if (a.head_dim == 64) hipLaunchKernelGGL(k_attn_decode_join<64>, jg, dim3(256), 0, st, a, grid);
    else if (a.head_dim == 128) hipLaunchKernelGGL(k_attn_decode_join<128>, jg, dim3(256), 0, st, a, grid);
    else hipLaunchKernelGGL(k_attn_decode_join<256>, jg, dim3(256), 0, st, a, grid);
    return hipGetLastError() == hipSuccess ? FP4_OK : FP4_ERR_HIP;
}

}  // namespace fp4k
