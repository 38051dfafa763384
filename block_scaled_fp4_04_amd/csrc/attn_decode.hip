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
// and the rescaling are rare; P stays below 2^8 (NVFP4: 2^15), which neither its 16-bit
// form nor the fp32 sums mind.  P is rounded to 16 bits (bf16, or f16 for NVFP4) because the matrix
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

constexpr int kTile = 128;          // keys of one work unit
constexpr int kOver = 1;            // what a row costs beside its tiles, in units
constexpr float kLazy = 8.0f;       // log2 headroom before the running maximum moves
// log2 by which the softmax weights of the f16 form (NVFP4) stand above 1 where the running maximum
// was taken: they stay below 2^15, and the smallest f16 is then 2^-31 of the largest weight rather
// than 2^-24, below which a weight would count in the softmax sum and be lost from the output
constexpr float kRaise = 7.0f;
// Past this running maximum the rounding of scale * score and of the maximum differ by enough to matter
// in exp2(fma(score, scale, -maximum)) (by a factor 2^(2^-4) here, by any factor beyond): the two are
// then rounded alike before they are subtracted.
constexpr float kFar = 0x1p20f;

constexpr int kv_bits(int fmt) { return fmt == FP4_KV_BF16 ? 16 : fmt == FP4_KV_MXFP8 ? 8 : 4; }
constexpr int kv_block(int fmt) { return fmt == FP4_KV_NVFP4 ? 16 : 32; }

// ------------------------------------------------------------ work split --

// First key a sequence's tiles start at (32-aligned) and the number of its tiles;
// an empty sequence has one (empty) tile, whose workgroup writes the zero row.
struct SeqSpan {
    int len, start, a0, tiles;
    __device__ __forceinline__ int cost() const { return tiles + kOver; }
};

// Block table and lengths are read through the constant address space: they do not
// change during the kernel, and a wave-uniform index then takes a scalar load.
typedef const __attribute__((address_space(4))) int32_t *const_i32;
__device__ __forceinline__ const_i32 as_const(const int32_t *p) { return (const_i32)(uintptr_t)p; }

__device__ __forceinline__ SeqSpan seq_span(const DecodeArgs &a, int b)
{
    SeqSpan s;
    int n = as_const(a.seq_lens)[b];
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

// What one row of every sequence costs, added up along the sequences.  A lane keeps the
// cost of sequence `lane` and the sum up to it; sequences past 64 are gone through again
// when one is looked for.
struct Plan {
    int cost, sum;    // of sequence `lane`, and of sequences 0 .. lane
    int head, total;  // of the first 64 sequences, and of all
};

__device__ __forceinline__ Plan make_plan(const DecodeArgs &a)
{
    const int lane = threadIdx.x & 63;
    Plan p;
    p.cost = lane < a.seqs ? seq_span(a, lane).cost() : 0;
    p.sum = wave_inclusive_sum(p.cost);
    p.head = p.total = __builtin_amdgcn_readlane(p.sum, 63);
    if (a.seqs > 64) {
        int more = 0;
        for (int b0 = 64; b0 < a.seqs; b0 += 64) more += b0 + lane < a.seqs ? seq_span(a, b0 + lane).cost() : 0;
        p.total += __builtin_amdgcn_readlane(wave_inclusive_sum(more), 63);
    }
    return p;
}

// The sequence at x (0 <= x < total) along the sum, and the sum before it.
__device__ __forceinline__ void find_seq(const DecodeArgs &a, const Plan &p, int x, int &b, int &before)
{
    const int lane = threadIdx.x & 63;
    int cost = p.cost, sum = p.sum, base = 0, b0 = 0;
    while (x >= base + __builtin_amdgcn_readlane(sum, 63) && b0 + 64 < a.seqs) {
        base += __builtin_amdgcn_readlane(sum, 63);
        b0 += 64;
        cost = b0 + lane < a.seqs ? seq_span(a, b0 + lane).cost() : 0;
        sum = wave_inclusive_sum(cost);
    }
    int i = __builtin_popcountll(__ballot(base + sum <= x));  // sequences that end at or before x
    i = i > 63 ? 63 : i;
    b = b0 + i;
    before = base + __builtin_amdgcn_readlane(sum - cost, i);
}

// The sum before sequence b.
__device__ __forceinline__ int cost_before(const DecodeArgs &a, const Plan &p, int b)
{
    if (b < 64) return __builtin_amdgcn_readlane(p.sum - p.cost, b);
    const int lane = threadIdx.x & 63;
    int more = 0;
    for (int b0 = 64; b0 < b; b0 += 64) more += b0 + lane < b ? seq_span(a, b0 + lane).cost() : 0;
    return p.head + __builtin_amdgcn_readlane(wave_inclusive_sum(more), 63);
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

// Waves of a workgroup, and waves a SIMD is to hold (which bounds the registers).
template <int FMT, int D, bool SPLIT>
struct Shape {
    static constexpr int kHold = D < 256 ? (D * kv_bits(FMT) <= 512 ? 4 : 3) : (FMT == FP4_KV_BF16 ? 1 : 2);
    static constexpr int kWaves = SPLIT || kHold == 1 ? 4 : 8;
    static constexpr int kPerCu = kHold * 4 / kWaves;  // workgroups a CU holds
};

// Orders LDS accesses of the workgroup; loads from memory stay in flight across it.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// SPLIT: the workgroups share all units; else one workgroup per row.
template <int FMT, int D, bool SPLIT>
__global__ __launch_bounds__((64 * Shape<FMT, D, SPLIT>::kWaves), (SPLIT ? Shape<FMT, D, SPLIT>::kHold : 1)) void k_attn_decode(DecodeArgs a)
{
    using C = Cfg<FMT, D>;
    constexpr int kWaves = Shape<FMT, D, SPLIT>::kWaves;
    constexpr int kStride = 32 * kWaves;  // keys the workgroup takes at a time
    static_assert(!SPLIT || kTile % kStride == 0, "a unit is a whole number of passes");
    __shared__ f32x4 sm_o[kWaves / 2][C::kDT][64];
    __shared__ float sm_m[kWaves][16], sm_l[kWaves][16];
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    const int rows = a.kv_heads * a.head_tiles;
    const int wg = blockIdx.x + (SPLIT ? 0 : a.first);
    int u = wg, u_end = wg + 1, b = 0, base = 0;
    SeqSpan sp;
    if constexpr (SPLIT) {
        const Plan plan = make_plan(a);
        const int units = plan.total * rows;
        const int grid = (int)gridDim.x < units ? (int)gridDim.x : units;
        if (wg >= grid) return;
        const Share sh = share_of(units, grid);
        u = share_start(sh, wg);
        u_end = share_start(sh, wg + 1);
        int before;
        find_seq(a, plan, u / rows, b, before);
        base = before * rows;  // first unit of sequence b
    } else {
        b = wg / rows;
    }
    sp = seq_span(a, b);
    // the lane's offsets from a sub-tile's first key
    const uint32_t k_lane = n * C::kRow + g * C::kKB, v_lane = 4 * g * C::kRow + n * C::kVB;
    const uint32_t ks_lane = ((g * C::kKV / C::kBlk) << a.page_shift) + n;
    const uint32_t vs_lane = ((n * C::kVV / C::kBlk) << a.page_shift) + 4 * g;
    // the next segment (a range of one row's tiles) of this workgroup's units; false when they are used up
    int r = 0, t0 = 0, t1 = 0;
    auto advance = [&]() -> bool {
        if constexpr (SPLIT) {
            while (u < u_end) {
                while (u >= base + sp.cost() * rows) {
                    base += sp.cost() * rows;
                    sp = seq_span(a, ++b);
                }
                // a row's units: kOver that stand for its fixed cost, then its tiles
                r = (u - base) / sp.cost();
                const int row_u = base + r * sp.cost(), first = u - row_u, left = u_end - row_u;
                t0 = first > kOver ? first - kOver : 0;
                t1 = left >= sp.cost() ? sp.tiles : left - kOver;
                u = row_u + sp.cost();
                if (t1 > t0) return true;  // else only (a part of) the fixed cost
            }
            return false;
        } else {
            const bool first = u < u_end;
            r = wg - b * rows;
            t0 = 0;
            t1 = sp.tiles;
            u = u_end;
            return first;
        }
    };

    // ---- raw bytes of 32 keys and of their values, fetched ahead of their use
    uint32_t kr[2][C::kKW], ksr[2][C::kScaled ? C::kKL * C::kKS : 1];
    uint32_t vr[8][C::kVL][C::kVW], vsr[2][C::kVL];
    uint4 q[C::kSteps];
    int hkv = 0, head0 = 0, nh = 0, key0 = 0, seg_end = 0;
    const int page_mask = (1 << a.page_shift) - 1;
    // pages of the two sub-tiles that are fetched next, looked up a pass ahead of their use; a
    // sub-tile past the sequence's end reads its last page (its keys are masked)
    int page_id[2];
    auto look_up = [&](int key0) {
        const const_i32 table = as_const(a.table + b * a.table_stride);
        const int top_page = (sp.len - 1) >> a.page_shift;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int page = (key0 + 16 * j) >> a.page_shift;
            page_id[j] = table[page < top_page ? page : top_page];
        }
    };
    // first row of a sub-tile's page within its pool, counted in tokens of one head
    auto block_of = [&](int j) -> int64_t {
        int id = page_id[j];
        id = id < 0 ? 0 : (id >= a.pages ? a.pages - 1 : id);
        return ((int64_t)id * a.kv_heads + hkv) << a.page_shift;
    };
    auto fetch_k = [&](int key0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t block = block_of(j);
            const int off = (key0 + 16 * j) & page_mask;
            const uint8_t *kp = a.k_codes + (block + off) * C::kRow;
#pragma unroll
            for (int i = 0; i < C::kKL; ++i) load_dwords<C::kKB>(kp + i * 4 * C::kKB + k_lane, &kr[j][i * (C::kKB / 4)]);
            if constexpr (C::kScaled) {
                const uint8_t *ksp = a.k_scales + block * (D / C::kBlk) + off;
#pragma unroll
                for (int i = 0; i < C::kKL; ++i)
#pragma unroll
                    for (int e = 0; e < C::kKS; ++e)
                        ksr[j][i * C::kKS + e] = (ksp + ((i * 4 * C::kKV / C::kBlk + e) << a.page_shift))[ks_lane];
            }
        }
    };
    auto fetch_v = [&](int key0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t block = block_of(j);
            const int off = (key0 + 16 * j) & page_mask;
            const uint8_t *vp = a.v_codes + (block + off) * C::kRow;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int h = 0; h < C::kVL; ++h) load_dwords<C::kVB>(vp + t * C::kRow + h * 16 * C::kVB + v_lane, vr[4 * j + t][h]);
            if constexpr (C::kScaled) {
                const uint8_t *vsp = a.v_scales + block * (D / C::kBlk) + off;
#pragma unroll
                for (int h = 0; h < C::kVL; ++h)
                    vsr[j][h] = *reinterpret_cast<const uint32_t *>(vsp + ((h * 16 * C::kVV / C::kBlk) << a.page_shift) + vs_lane);
            }
        }
    };
    // a segment's query heads (the B operand: lane n = head, the same order of d as K's
    // loads), first keys and first values, requested before the segment before it is joined
    auto begin = [&]() {
        hkv = r / a.head_tiles;
        const int h0 = (r - hkv * a.head_tiles) * 16;
        nh = a.group - h0 < 16 ? a.group - h0 : 16;
        head0 = hkv * a.group + h0;
        key0 = sp.a0 + t0 * kTile + wave * 32;
        if (sp.len > 0) look_up(key0);
        seg_end = sp.a0 + t1 * kTile < sp.len ? sp.a0 + t1 * kTile : sp.len;
        const uint16_t *qp = a.q + b * a.q_seq + (int64_t)(head0 + n) * a.q_head;
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s) {
            const int i = 8 * s / C::kKV, e = 8 * s % C::kKV;
            q[s] = make_uint4(0, 0, 0, 0);
            if (n < nh) q[s] = *reinterpret_cast<const uint4 *>(qp + i * 4 * C::kKV + g * C::kKV + e);
        }
        if (key0 < seg_end) {
            fetch_k(key0);
            fetch_v(key0);
            look_up(key0 + kStride);
        }
    };

    bool more = advance();
    if (more) begin();
    while (more) {
        float c = a.scale_log2;
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
        c = fmaxf(c, 0x1p-140f);  // a scale of 0: -inf of a masked key stays -inf, every other score becomes 0

        f32x4 o[C::kDT];
#pragma unroll
        for (int i = 0; i < C::kDT; ++i) o[i] = f32x4{0, 0, 0, 0};
        constexpr float kUp = C::kF16 ? kRaise : 0.0f;
        float m = -INFINITY, l = 0.0f;  // m: the running maximum less kUp
        bool far = false;               // of any head of the wave

        // scores of the 32 keys in kr: s[j] holds keys 16 j + 4 g .. + 3 of head n
        auto scores = [&](f32x4 (&s)[2]) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                s[j] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int st = 0; st < C::kSteps; ++st) {
                    const int i = 8 * st / C::kKV, e = 8 * st % C::kKV;
                    const uint32_t sc = C::kScaled ? ksr[j][i * C::kKS + e / C::kBlk] : 0;
                    s[j] = mfma16<C::kF16>(widen8<FMT>(&kr[j][8 * st * C::kBits / 32], sc), q[st], s[j]);
                }
            }
        };
        // keys out of range: no score, and their values (which may be anything) become 0
        auto mask_scores = [&](int key, f32x4 (&s)[2]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = key + 16 * (i >> 2) + 4 * g + (i & 3);
                s[i >> 2][i & 3] = k >= sp.start && k < sp.len ? s[i >> 2][i & 3] : -INFINITY;
            }
        };
        auto mask_values = [&](int key) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = key + 16 * (i >> 2) + 4 * g + (i & 3);
                const bool in = k >= sp.start && k < sp.len;
#pragma unroll
                for (int h = 0; h < C::kVL; ++h) {
#pragma unroll
                    for (int w = 0; w < C::kVW; ++w) vr[i][h][w] = in ? vr[i][h][w] : 0u;
                    if constexpr (C::kScaled)
                        vsr[i >> 2][h] = in ? vsr[i >> 2][h] : vsr[i >> 2][h] & ~(0xFFu << (8 * (i & 3)));
                }
            }
        };
        // softmax weights of the scores, as the B operand of O
        auto weights = [&](f32x4 (&s)[2]) -> uint4 {
            const float tm = c * fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                                       fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
            if (__ballot(tm > m + (kUp + kLazy))) {
                const float mn = fmaxf(m, xor16_max(tm) - kUp);
                const float alpha = mn == m ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
                m = mn;
                l *= alpha;
#pragma unroll
                for (int i = 0; i < C::kDT; ++i) o[i] *= alpha;
                far = __ballot(m > -INFINITY && __builtin_fabsf(m) > kFar) != 0;
            }
            float mm = m == -INFINITY ? 0.0f : -m, cs = c;
            if (far) {
#pragma clang fp contract(off)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float t = s[i >> 2][i & 3] * c;
                    s[i >> 2][i & 3] = t + mm;
                }
                cs = 1.0f;
                mm = 0.0f;
            }
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i >> 2][i & 3], cs, mm));
            l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
            return make_uint4(pack2<C::kF16>(p[0], p[1]), pack2<C::kF16>(p[2], p[3]), pack2<C::kF16>(p[4], p[5]),
                              pack2<C::kF16>(p[6], p[7]));
        };
        // O^T: a pair of d at a time, its two rows of V^T gathered from the 8 keys
        auto values = [&](const uint4 &pf) {
#pragma unroll
            for (int h = 0; h < C::kVL; ++h)
#pragma unroll
                for (int pr = 0; pr < C::kVV / 2; ++pr) {
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        w[i] = widen_pair<FMT>(vr[i][h], pr, C::kScaled ? (vsr[i >> 2][h] >> (8 * (i & 3))) & 0xFFu : 0u);
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

        if (key0 < seg_end) {
            f32x4 s[2];
            // the next keys are requested as soon as this pass's keys are used up, the next
            // values as soon as its values are: one set of registers, loads always in flight
            for (; key0 + kStride < seg_end; key0 += kStride) {
                scores(s);
                fetch_k(key0 + kStride);
                __builtin_amdgcn_sched_barrier(0);
                const bool cut = key0 < sp.start;  // (a further pass follows, so the end is not cut)
                if (cut) mask_scores(key0, s);
                const uint4 pf = weights(s);
                if (cut) mask_values(key0);
                values(pf);
                fetch_v(key0 + kStride);
                look_up(key0 + 2 * kStride);
                __builtin_amdgcn_sched_barrier(0);
            }
            scores(s);
            const bool cut = key0 < sp.start || key0 + 32 > sp.len;
            if (cut) mask_scores(key0, s);
            const uint4 pf = weights(s);
            if (cut) mask_values(key0);
            values(pf);
        }

        // ---- the waves' results become one, while the next segment's first loads are in flight
        const int e_b = b, e_head0 = head0, e_nh = nh, e_hkv = hkv, slot = 2 * wg + (t0 == 0);
        const bool whole = t0 == 0 && t1 == sp.tiles;
        more = advance();
        if (more) begin();
        __builtin_amdgcn_sched_barrier(0);
        l = xor16_sum(l);
        if (lane < 16) {
            sm_m[wave][n] = m;
            sm_l[wave][n] = l;
        }
        lds_barrier();
        float M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) M = fmaxf(M, sm_m[w][n]);
        const float Ms = M == -INFINITY ? 0.0f : M;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) L += sm_l[w][n] * __builtin_amdgcn_exp2f(sm_m[w][n] - Ms);
        const float beta = __builtin_amdgcn_exp2f(m - Ms);
#pragma unroll
        for (int i = 0; i < C::kDT; ++i) o[i] *= beta;
#pragma unroll
        for (int half = kWaves / 2; half >= 1; half >>= 1) {
            if (wave >= half && wave < 2 * half) {
#pragma unroll
                for (int i = 0; i < C::kDT; ++i) sm_o[wave - half][i][lane] = o[i];
            }
            lds_barrier();
            if (wave < half) {
#pragma unroll
                for (int i = 0; i < C::kDT; ++i) o[i] += sm_o[wave][i][lane];
            }
            if (half > 1) lds_barrier();
        }
        if (wave == 0 && n < e_nh) {
            float *po = nullptr;
            float f = 1.0f;
            if (whole) {
                f = L == 0.0f ? 0.0f : 1.0f / L;
                if constexpr (C::kF16) f *= a.v_tscale[e_hkv];
                if (a.lse && g == 0) a.lse[(int64_t)e_b * a.heads + e_head0 + n] = (M + __builtin_amdgcn_logf(L)) * 0.69314718f;
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
                            uint16_t *p = reinterpret_cast<uint16_t *>(a.out) + e_b * a.o_seq + (e_head0 + n) * a.o_head + d + i;
                            *reinterpret_cast<uint2 *>(p) = make_uint2(pack2<false>(v.x, v.y), pack2<false>(v.z, v.w));
                        } else {
                            float *p = reinterpret_cast<float *>(a.out) + e_b * a.o_seq + (e_head0 + n) * a.o_head + d + i;
                            *reinterpret_cast<float4 *>(p) = v;
                        }
                    }
                }
        }
        if (more) lds_barrier();  // the next segment writes sm_m, sm_l and sm_o again
    }
}

// One workgroup per (sequence, query head): adds up the partial results of a row
// that several workgroups of k_attn_decode share.  Four d a thread, the partial
// results dealt to 4 THREADS / D groups of threads.
template <int D, int THREADS>
__global__ __launch_bounds__(THREADS) void k_attn_decode_join(DecodeArgs a, int grid_full)
{
    constexpr int kLanes = D / 4, kParts = THREADS / kLanes;
    __shared__ f32x4 sm[kParts][kLanes];
    __shared__ float sm_m[kParts], sm_l[kParts];
    const int row = blockIdx.x + a.first, b = row / a.heads, head = row - b * a.heads;
    const int hkv = head / a.group, hg = head - hkv * a.group, n = hg & 15;
    const int rows = a.kv_heads * a.head_tiles;
    const Plan plan = make_plan(a);
    const int units = plan.total * rows;
    const int grid = grid_full < units ? grid_full : units;
    const Share sh = share_of(units, grid);
    const SeqSpan sp = seq_span(a, b);
    const int r = hkv * a.head_tiles + (hg >> 4);
    const int u0 = cost_before(a, plan, b) * rows + r * sp.cost() + kOver;  // its first tile
    const int w0 = share_owner(sh, u0), w1 = share_owner(sh, u0 + sp.tiles - 1);
    if (w0 == w1) return;
    const int d = threadIdx.x % kLanes, part = threadIdx.x / kLanes;
    f32x4 acc = {0, 0, 0, 0};
    float m = -INFINITY, L = 0.0f;
#pragma unroll 4
    for (int w = w0 + part; w <= w1; w += kParts) {
        const int64_t i = (int64_t)(2 * w + (w == w0)) * a.part_heads + n;
        const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + i * 2);
        const f32x4 o = *reinterpret_cast<const f32x4 *>(a.part_o + i * D + 4 * d);
        const float mn = fmaxf(m, ml.x), ms = mn == -INFINITY ? 0.0f : mn;
        const float fa = __builtin_amdgcn_exp2f(m - ms), fb = __builtin_amdgcn_exp2f(ml.x - ms);
        L = L * fa + ml.y * fb;
        acc = acc * fa + o * fb;
        m = mn;
    }
    if (d == 0) sm_m[part] = m;
    __syncthreads();
    float M = sm_m[0];
#pragma unroll
    for (int i = 1; i < kParts; ++i) M = fmaxf(M, sm_m[i]);
    const float f0 = __builtin_amdgcn_exp2f(m - (M == -INFINITY ? 0.0f : M));
    acc *= f0;
    L *= f0;
    sm[part][d] = acc;
    if (d == 0) sm_l[part] = L;
    __syncthreads();
    if (part != 0) return;
    L = sm_l[0];
#pragma unroll
    for (int i = 1; i < kParts; ++i) {
        acc += sm[i][d];
        L += sm_l[i];
    }
    float f = L == 0.0f ? 0.0f : 1.0f / L;
    if (a.v_tscale) f *= a.v_tscale[hkv];
    acc *= f;
    const int64_t p = b * a.o_seq + head * a.o_head + 4 * d;
    if (a.out_bf16)
        *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(a.out) + p) = make_uint2(pack2<false>(acc[0], acc[1]), pack2<false>(acc[2], acc[3]));
    else
        *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(a.out) + p) = acc;
    if (a.lse && d == 0) a.lse[(int64_t)b * a.heads + head] = (M + __builtin_amdgcn_logf(L)) * 0.69314718f;
}

int64_t decode_units_bound(int64_t seqs, int64_t kv_heads, int64_t head_tiles, int64_t max_len)
{
    return seqs * kv_heads * head_tiles * ((max_len + 31 + kTile - 1) / kTile + kOver);
}

// Whether rows are split among workgroups: not when a row's longest context is a few
// passes of one workgroup, whose latency is below that of a second launch (one launch / split: 8 bf16 rows of
// 600 keys 9.8 / 13.6 us, 1000 13.2 / 13.5, 1900 20.8 / 13.3; 128 NVFP4 rows of 600 9.5 / 13.5, 1000 10.9 / 15.3,
// 1900 14.9 / 17.4).
static bool decode_splits(int64_t max_len) { return max_len > 1024; }

// Workgroups of a split launch: as many as the device holds at once.
int decode_grid(int64_t seqs, int64_t kv_heads, int64_t head_tiles, int64_t max_len)
{
    if (!decode_splits(max_len)) return 0;
    const int64_t units = decode_units_bound(seqs, kv_heads, head_tiles, max_len);
    const int64_t most = 4 * (int64_t)device_cu_count();  // at most 4 workgroups a CU (Shape::kPerCu)
    return (int)(units < most ? units : most);
}

// Launches `kernel` over `blocks` workgroups, as several launches where one would pass the 2^32 threads of
// a launch; a.first is then the first workgroup of each.
template <typename Kernel>
static void launch_rows(Kernel kernel, DecodeArgs a, int64_t blocks, int threads, hipStream_t st, int arg = 0)
{
    const int64_t most = (int64_t(1) << 31) / threads;
    for (int64_t first = 0; first < blocks; first += most) {
        a.first = (int)first;
        kernel(a, dim3((unsigned)(blocks - first < most ? blocks - first : most)), dim3(threads), st, arg);
    }
}

template <int FMT, int D>
static void launch_decode(const DecodeArgs &a, hipStream_t st)
{
    using S = Shape<FMT, D, true>;
    const int rows = a.kv_heads * a.head_tiles;
    // a window bounds every row alike: where the rows fill the chip, one launch serves it as well
    // (129 sequences, window 1024, head_dim 256: 28.0 -> 21.5 us; 64 of 8000 keys, window 2000: 33.5 -> 26.3 us;
    // window 4096: 57.7 -> 50.7 us, but on a ragged batch of 128 46.5 -> 57.0 us)
    const int64_t reach = a.window > 0 && a.window + 31 < a.max_len ? a.window + 31 : a.max_len;
    // every workgroup of the two launches adds up all lengths, which with this many sequences costs more than
    // the longest row can gain (sequences, keys of the table: 512, 2048: 48.4 -> 43.8 us; 4096, 2048: 381 -> 242;
    // 8192, 2048: 357 -> 84; one long row among short ones breaks even at 256, 2048 and 512, 4096)
    const bool many = 4 * (int64_t)a.seqs >= a.max_len;
    if (!decode_splits(reach) || many || (a.window > 0 && reach <= 2100 && a.seqs * rows >= device_cu_count())) {
        launch_rows([](const DecodeArgs &x, dim3 g, dim3 t, hipStream_t s, int) {
            hipLaunchKernelGGL((k_attn_decode<FMT, D, false>), g, t, 0, s, x);
        }, a, (int64_t)a.seqs * rows, 64 * Shape<FMT, D, false>::kWaves, st);
        return;
    }
    const int64_t units = decode_units_bound(a.seqs, a.kv_heads, a.head_tiles, a.max_len);
    const int64_t most = S::kPerCu * (int64_t)device_cu_count();
    const int grid = (int)(units < most ? units : most);
    hipLaunchKernelGGL((k_attn_decode<FMT, D, true>), dim3(grid), dim3(64 * S::kWaves), 0, st, a);
    // a wave a row where there are many (their parts are few), else four (whole calls, four waves / one: 2560 rows
    // 47.7 / 45.6 us, 2048 25.8 / 23.4, 1280 45.4 / 45.6, 256 16.3 / 17.2, 96 long ones 45.8 / 49.0)
    const int64_t jrows = (int64_t)a.seqs * a.heads;
    if (jrows > 1024)
        launch_rows([](const DecodeArgs &x, dim3 g, dim3 t, hipStream_t s, int grid) {
            hipLaunchKernelGGL((k_attn_decode_join<D, 64>), g, t, 0, s, x, grid);
        }, a, jrows, 64, st, grid);
    else hipLaunchKernelGGL((k_attn_decode_join<D, 256>), dim3((unsigned)jrows), dim3(256), 0, st, a, grid);
}

template <int FMT>
static void launch_fmt(const DecodeArgs &a, hipStream_t st)
{
    if (a.head_dim == 64) launch_decode<FMT, 64>(a, st);
    else if (a.head_dim == 128) launch_decode<FMT, 128>(a, st);
    else launch_decode<FMT, 256>(a, st);
}

fp4_status launch_attn_decode(const DecodeArgs &a, fp4_kv_format fmt, hipStream_t st)
{
    if (fmt == FP4_KV_BF16) launch_fmt<FP4_KV_BF16>(a, st);
    else if (fmt == FP4_KV_MXFP8) launch_fmt<FP4_KV_MXFP8>(a, st);
    else if (fmt == FP4_KV_NVFP4) launch_fmt<FP4_KV_NVFP4>(a, st);
    else launch_fmt<FP4_KV_MXFP4>(a, st);
    return hipGetLastError() == hipSuccess ? FP4_OK : FP4_ERR_HIP;
}

}  // namespace fp4k
