// attn_prefill.hip -- attention of whole prompts: packed sequences of different
// lengths, grouped heads, causal and windowed masks.
//
// For query token i of a sequence with lq queries and lk keys, at position
// pos = i + lk - lq (the last query stands at the last key), and query head h:
//   t_j = scale q.k_j over the keys j that i sees, o = sum_j exp(t_j - lse) v_j,
//   lse = log sum_j exp(t_j);  j < lk, j <= pos (causal), j > pos - window (window > 0).
//
// Bound: 4 D flop a (query head, key) pair on the matrix core; K and V are read once
// per row tile from L2, so for long prompts the MFMA rate is the floor.
//
// Rows of a tile are (token, head of the group) pairs, numbered token-major, so every
// group size fills the tiles, a tile covers few tokens (little of it is masked) and K
// and V are staged once for all heads of the group.
//
// One wave, 32 rows, 64 keys at a time, 32x32x16 MFMA:
//   S^T = K Q^T  rows = keys, columns = query rows: a lane holds, for its one query row
//                lane & 31, the keys 8 a + 4 h + i of each 32 (h = lane >> 5, a, i < 4).
//                Row statistics then need one exchange, between the wave's halves.
//   O^T += V^T P^T  the contracted keys are numbered so that slot (h, j) of step s is
//                the key the lane already holds (16 s + 8 (j >> 2) + 4 h + (j & 3)): P
//                goes from the softmax to the matrix core without leaving its lane.
//                V^T comes from row-major V in LDS by transposing LDS reads (4 keys x
//                16 d per 16 lanes).
// K and V tiles go to LDS by direct copies (two buffers, the next tile in flight while
// one is used); 16-byte chunks are XOR-swizzled by row so that neither kind of read
// meets a bank twice in a phase.
#include "device_common.h"
#include "internal.h"

namespace fp4k {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;

namespace {

constexpr int kRows = 128;     // rows of a workgroup: four waves of 32
constexpr float kLazy = 8.0f;  // log2 headroom before the running maximum moves
// Past this running maximum the rounding of scale * score and of the maximum differ by enough to matter
// in exp2(fma(score, scale, -maximum)) (by a factor 2^(2^-4) here, by any factor beyond): the two are
// then rounded alike before they are subtracted.
constexpr float kFar = 0x1p20f;

// A row tile: its sequence (-1: past the last), its number there, and the sequence's rows,
// clamped into the buffers.
struct QTile {
    int b, tile;
    int q0, lq, k0, lk;
};

__device__ __forceinline__ int clamp_offset(int v, int64_t top) { return v < 0 ? 0 : ((int64_t)v > top ? (int)top : v); }

// More sequences than this are not counted through by every workgroup, but searched (find_slot): of 1 to 4 tokens
// each, 257 take 12.4 us either way, 512 14.9 -> 12.9 us, 4096 322 -> 79 us, 16384 4186 -> 315 us.
constexpr int kManySeqs = 256;

// Row tile x where each sequence has a tile to spare: sequence b's tiles begin at
// floor(cu_q[b] group / kRows) + b, which leaves room for all of them and is found by search, 64
// sequences at a time.
__device__ __forceinline__ QTile find_slot(const PrefillArgs &a, int x)
{
    const int lane = threadIdx.x & 63;
    auto start = [&](int b) { return (int)((int64_t)clamp_offset(a.cu_q[b], a.q_tokens) * a.group / kRows) + b; };
    int lo = 0, span = a.seqs;  // the answer is in [lo, lo + span)
    while (span > 1) {
        const int step = (span + 63) >> 6;
        const bool past = lane * step < span && start(lo + lane * step) <= x;
        const int n = __builtin_popcountll(__ballot(past));
        const int skip = n > 0 ? (n - 1) * step : 0;
        lo += skip;
        span = span - skip < step ? span - skip : step;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    const int q0 = clamp_offset(a.cu_q[lo], a.q_tokens), q1 = clamp_offset(a.cu_q[lo + 1], a.q_tokens);
    const int k0 = clamp_offset(a.cu_k[lo], a.k_tokens), k1 = clamp_offset(a.cu_k[lo + 1], a.k_tokens);
    const int lq = q1 > q0 ? q1 - q0 : 0, tiles = (int)(((int64_t)lq * a.group + kRows - 1) / kRows);
    const int t = x - start(lo);
    if (t < 0 || t >= tiles) return {-1, 0, 0, 0, 0, 0};
    return {lo, tiles - 1 - t, q0, lq, k0, k1 > k0 ? k1 - k0 : 0};
}

// Row tile x of the concatenated sequences, a sequence's last tiles first: they see the most
// keys.  (The longest sequence first as well gained nothing measurable and costs a pass
// over the lanes.)  Where the chip holds all workgroups at once, two a CU, the second half
// comes in reverse: the CUs that got the longest tiles first get the shortest ones as
// their second (2048 tokens, 32/8 heads of 128: 48.4 -> 47.5 us; two prompts of 1000: 34.3 -> 28.9 us).
__device__ __forceinline__ QTile find_tile(const PrefillArgs &a, int x)
{
    if (a.seqs > kManySeqs) return find_slot(a, x);
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += 64) {
        const int b = b0 + lane < a.seqs ? b0 + lane : a.seqs - 1;
        const int q0 = clamp_offset(a.cu_q[b], a.q_tokens), q1 = clamp_offset(a.cu_q[b + 1], a.q_tokens);
        const int k0 = clamp_offset(a.cu_k[b], a.k_tokens), k1 = clamp_offset(a.cu_k[b + 1], a.k_tokens);
        const int lq = b0 + lane < a.seqs && q1 > q0 ? q1 - q0 : 0;
        const int t = (int)(((int64_t)lq * a.group + kRows - 1) / kRows);
        int inc = t;
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(inc, off, kWave);
            if (lane >= off) inc += o;
        }
        const int sum = __builtin_amdgcn_readlane(inc, 63);
        if (a.seqs <= 64 && x >= a.fold_at && x < sum && sum * a.kv_heads <= a.fold_most) x = sum - 1 - (x - a.fold_at);
        if (x < base + sum) {
            int i = __builtin_popcountll(__ballot(base + inc <= x));
            i = i > 63 ? 63 : i;
            QTile r;
            r.b = b0 + i;
            r.tile = base + __builtin_amdgcn_readlane(inc, i) - 1 - x;
            r.q0 = __builtin_amdgcn_readlane(q0, i);
            r.lq = __builtin_amdgcn_readlane(lq, i);
            r.k0 = __builtin_amdgcn_readlane(k0, i);
            r.lk = __builtin_amdgcn_readlane(k1 > k0 ? k1 - k0 : 0, i);
            return r;
        }
        base += sum;
    }
    return {-1, 0, 0, 0, 0, 0};
}

// The keys [lo, hi) that the rows of a tile see, `lo` rounded down to a tile of keys, and the parts they
// are cut into, of a.splits at most: as many as parts of kPartKeys make, so that a row tile with few keys
// among longer ones (or behind a window) has one part, which writes the output itself.  (Four chunks of
// 33 tokens behind 6000 keys: parts of 256 keys 36.9 us, 448 33.4, 512 32.0, all 32 splits 41.8; sixteen of up
// to 300 behind 2000: 30.1, 30.1, 31.5, 29.6.)
constexpr int kPartKeys = 448;
struct KeyRange {
    int lo, hi, parts;
};
template <int KEYS>
__device__ __forceinline__ KeyRange key_range(const PrefillArgs &a, const QTile &qt)
{
    const uint32_t rows = (uint32_t)qt.lq * (uint32_t)a.group, row0 = (uint32_t)qt.tile * kRows;
    const int first = (int)(row0 / (uint32_t)a.group) + qt.lk - qt.lq;  // position of the first row
    const int last = (int)((row0 + kRows < rows ? row0 + kRows - 1 : rows - 1) / (uint32_t)a.group) + qt.lk - qt.lq;
    KeyRange k;
    k.lo = (a.window > 0 && first - a.window + 1 > 0 ? first - a.window + 1 : 0) & ~(KEYS - 1);
    k.hi = a.causal ? last + 1 : qt.lk;
    const int most = (k.hi - k.lo + kPartKeys - 1) / kPartKeys;
    k.parts = most < a.splits ? (most < 1 ? 1 : most) : a.splits;
    return k;
}

// swizzle of the 16-byte chunks of an LDS row
template <int D>
__device__ __forceinline__ int swz_k(int row)
{
    return D == 64 ? (row >> 1) & 7 : row & 15;
}
template <int D>
__device__ __forceinline__ int swz_v(int row)
{
    return D == 64 ? (row & 2) << 1 : (row & 3) << 2;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const bf16x2 v = {(__bf16)lo, (__bf16)hi};
    uint32_t r;
    __builtin_memcpy(&r, &v, 4);
    return r;
}

__device__ __forceinline__ float other_half(float v)
{
    return __shfl_xor(v, 32, kWave);
}

}  // namespace

template <int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_attn_prefill(PrefillArgs a)
{
    constexpr int kKeys = D == 256 ? 32 : 64;  // keys of a tile
    constexpr int kSub = kKeys / 32;
    constexpr int kRowB = 2 * D;             // bytes of an LDS row
    constexpr int kTileB = kKeys * kRowB;    // bytes of a tile of K or V
    constexpr int kCopies = kTileB / 4096;   // 1 KiB copies per wave and tile
    constexpr int kSteps = D / 16;           // MFMA steps of S
    constexpr int kDT = D / 32;              // MFMA tiles of O
    // Two buffers each for K and V, as objects of their own: the compiler then knows that a
    // copy into one does not touch the others, and does not wait for it at every LDS read.
    __shared__ __align__(16) uint8_t sm_k0[kTileB], sm_k1[kTileB], sm_v0[kTileB], sm_v1[kTileB];
    __shared__ uint32_t sm_found[2][4];  // by buffer of V and wave: infinities or NaN in what the wave has copied
    const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // blocks: (row tile, part, key head), the key head fastest
    const int block = blockIdx.x + a.first, xs = block / a.kv_heads, hkv = block - xs * a.kv_heads;
    const int x = xs / a.splits, split = xs - x * a.splits;
    const QTile qt = find_tile(a, x);
    if (qt.b < 0) return;

    const int64_t q0 = qt.q0, k0 = qt.k0;
    const int lq = qt.lq, lk = qt.lk;
    const int64_t rows = (int64_t)lq * a.group;
    const int64_t row0 = (int64_t)qt.tile * kRows;

    // this lane's row
    int64_t row = row0 + wave * 32 + col;
    const bool live = row < rows;
    if (!live) row = rows - 1;
    const int tok = (int)((uint32_t)row / (uint32_t)a.group), hg = (int)row - tok * a.group;
    const int head = hkv * a.group + hg;
    const int pos = tok + lk - lq;
    const int ub = a.causal ? pos + 1 : lk;                                  // keys [lb, ub)
    const int lb = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
    // the range of keys of the workgroup
    auto tok_of = [&](int64_t r) { return (int)((uint32_t)(r < rows ? r : rows - 1) / (uint32_t)a.group); };
    auto ub_of = [&](int t) { return a.causal ? t + lk - lq + 1 : lk; };
    auto lb_of = [&](int t) { const int p = t + lk - lq; return a.window > 0 && p - a.window + 1 > 0 ? p - a.window + 1 : 0; };
    const int g_full_hi = ub_of(tok_of(row0)), g_full_lo = lb_of(tok_of(row0 + kRows - 1));  // every row of the workgroup
    const KeyRange range = key_range<kKeys>(a, qt);
    int lo = range.lo, hi = range.hi;
    if (range.parts > 1) {
        const int share = ((hi - lo + kKeys - 1) / kKeys + range.parts - 1) / range.parts * kKeys;
        lo += split * share;
        hi = lo + share < hi ? lo + share : hi;
    }
    if (split >= range.parts) return;

    // ---- Q: the B operand, held for the whole tile
    uint4 q[kSteps];
    auto load_q = [&]() __attribute__((always_inline)) {
        const uint16_t *qp = a.q + (q0 + tok) * a.q_tok + head * a.q_head + 8 * half;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) q[s] = *reinterpret_cast<const uint4 *>(qp + 16 * s);
    };

    f32x16 o[kDT];
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
    float m = -INFINITY, l = 0.0f;

    // K and V tiles go to LDS through a descriptor that ends with the sequence's last row: rows
    // past it arrive as zeros.  The whole offset of a row is the lane's: the range check then
    // compares it with the descriptor's size alone.  (A row in the scalar offset is taken off the
    // size first, which a copy wholly past the end would bring below zero.)  A wave's copies are
    // kStep rows apart, which leaves their swizzle alone (D = 256: alternates it).
    constexpr int kStep = 4096 / kRowB;
    constexpr int kOfs = D == 256 ? 2 : 1;
    uint32_t k_ofs[kOfs], v_ofs[kOfs];
#pragma unroll
    for (int i = 0; i < kOfs; ++i) {
        const int r = (wave * 1024 + lane * 16) / kRowB, slot = (lane * 16 % kRowB) / 16;  // row of a copy, chunk
        k_ofs[i] = (uint32_t)(r * (int)a.k_tok + (slot ^ swz_k<D>(i * kStep + r)) * 8) * 2;
        v_ofs[i] = (uint32_t)(r * (int)a.v_tok + (slot ^ swz_v<D>(i * kStep + r)) * 8) * 2;
    }
    const uint16_t *kb = a.k + k0 * a.k_tok + hkv * a.k_head;
    const uint16_t *vb = a.v + k0 * a.v_tok + hkv * a.v_head;
    auto stage = [&](const uint16_t *base, int tok, const uint32_t (&ofs)[kOfs], int key0, uint8_t *dst)
                     __attribute__((always_inline)) {
        const int n = lk - key0 < kKeys ? lk - key0 : kKeys;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(base + key0 * (int64_t)tok),
                                                                           (short)0, ((n - 1) * tok + D) * 2, 0x00020000);
        int step = kStep * tok * 2;
        if constexpr (D == 256) asm volatile("" : "+s"(step));  // the sums are formed here, not kept in registers (which spill)
#pragma unroll
        for (int j = 0; j < kCopies; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(dst + wave * 1024 + j * 4096), 16,
                                                     (int)(ofs[j % kOfs] + (uint32_t)(j * step)), 0, 0, 0);
    };
    auto stage_k = [&](int key0, uint8_t *dst) __attribute__((always_inline)) { stage(kb, (int)a.k_tok, k_ofs, key0, dst); };
    auto stage_v = [&](int key0, uint8_t *dst) __attribute__((always_inline)) { stage(vb, (int)a.v_tok, v_ofs, key0, dst); };

    const float c = fmaxf(a.scale_log2, 0x1p-140f);  // a scale of 0: a masked key's -inf stays
    const int c16 = lane & 15, dgrp = (lane >> 4) & 1;
    auto scores = [&](const uint8_t *kt, f32x16 (&s)[kSub]) __attribute__((always_inline)) {
        const uint8_t *kr = kt + col * kRowB;
        int first = half ^ swz_k<D>(col);  // this lane's chunk of step 0
        if constexpr (D == 256) asm volatile("" : "+v"(first));  // the other steps' are formed here, not kept (which spills)
#pragma unroll
        for (int e = 0; e < 16 * kSub; ++e) s[e >> 4][e & 15] = 0.0f;
#pragma unroll
        for (int st = 0; st < kSteps; ++st)
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
                // (the swizzle acts on the low four bits of a chunk's number: beyond, a constant offset)
                const uint4 f = *reinterpret_cast<const uint4 *>(kr + 32 * j * kRowB + (st >> 3) * 256 + ((first ^ (2 * st & 15)) * 16));
                s[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(f), as_bf16x8(q[st]), s[j], 0, 0, 0);
            }
    };
    uint64_t far = 0;  // lanes whose |m| is past kFar: with any, settle() scales the scores and takes m off
    // A tile that some row of the workgroup does not see whole may hold infinities and NaN in keys that are masked
    // there, and the product would carry them into every row (0 times them is NaN).  Each wave therefore searches
    // what it has copied of such a tile before the barrier that hands it over; what is found is cleared in LDS,
    // and added to the rows that see it at the end, from memory.  (8192 tokens 652 -> 656 us, a windowed chunk
    // 312 -> 317 us, packed prompts 56.0 -> 55.9 us on one card; searched after the barrier, by every wave, in a
    // branch of its own 658, 319 and 56.9 us; a loop of its own for the whole tiles 681, 383 and 56.9 us.)
    auto clean = [&](int key0) { return __builtin_expect(key0 >= g_full_lo && key0 + kKeys <= g_full_hi, 1); };
    auto search = [&](const uint8_t *vt, uint32_t (&found)[4]) __attribute__((always_inline)) {
        __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xF << 8));  // vmcnt(0): the wave's own copies have arrived
        u16x2 top = {0, 0};
#pragma unroll
        for (int j = 0; j < kCopies; ++j) {
            const u32x4 w = *reinterpret_cast<const u32x4 *>(vt + wave * 1024 + j * 4096 + lane * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t x = w[e] & 0x7FFF7FFFu;
                u16x2 h;
                __builtin_memcpy(&h, &x, 4);
                top = __builtin_elementwise_max(top, h);
            }
        }
        const uint64_t any = __ballot(top[0] >= 0x7F80 || top[1] >= 0x7F80);
        if (lane == 0) found[wave] = any != 0;
    };
    // masks the scores of tile key0, whose values are in vt, and moves the running maximum
    auto settle = [&](int key0, f32x16 (&s)[kSub], const uint8_t *vt, uint32_t (&found)[4]) __attribute__((always_inline)) {
        if (!clean(key0)) {
            search(vt, found);
            // of the lane's keys 8 x + 4 half + i, those in [lb, ub)
            const int first = lb - key0 - 4 * half, last = ub - key0 - 4 * half;
#pragma unroll
            for (int j = 0; j < kSub; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int key = 32 * j + 8 * (e >> 2) + (e & 3);
                    s[j][e] = key >= first && key < last ? s[j][e] : -INFINITY;
                }
        }
        float tm = s[0][0];
#pragma unroll
        for (int e = 1; e < 16 * kSub; ++e) tm = fmaxf(tm, s[e >> 4][e & 15]);
        tm *= c;
        if (__ballot(tm > m + kLazy) | far) {
            const float mn = fmaxf(m, fmaxf(tm, other_half(tm)));
            const float alpha = mn == m ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= alpha;
#pragma unroll
            for (int i = 0; i < kDT; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[i][e] *= alpha;
            far = __ballot(m > -INFINITY && __builtin_fabsf(m) > kFar);
            if (far) {
#pragma clang fp contract(off)
                const float less = m == -INFINITY ? 0.0f : m;
#pragma unroll
                for (int e = 0; e < 16 * kSub; ++e) {
                    const float t = s[e >> 4][e & 15] * c;
                    s[e >> 4][e & 15] = t - less;
                }
            }
        }
    };
    // P of step st: keys 16 st + 8 (j >> 2) + 4 half + (j & 3), registers 8 (st & 1) .. + 7 of s[st >> 1]
    auto weights = [&](const f32x16 (&s)[kSub], uint4 (&p)[2 * kSub]) __attribute__((always_inline)) {
        const float cs = far ? 1.0f : c, mm = far || m == -INFINITY ? 0.0f : -m;
#pragma unroll
        for (int st = 0; st < 2 * kSub; ++st) {
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[st >> 1][8 * (st & 1) + i], cs, mm));
            l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
            p[st] = make_uint4(pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]), pack_bf16(e[4], e[5]), pack_bf16(e[6], e[7]));
        }
    };
    // V^T: lane c of a 16-lane group addresses key c >> 2 of 4, d 4 (c & 3) of 16
    auto values = [&](const uint8_t *vt, const uint4 (&p)[2 * kSub]) __attribute__((always_inline)) {
#pragma unroll
        for (int st = 0; st < 2 * kSub; ++st)
#pragma unroll
            for (int i = 0; i < kDT; ++i) {
                uint4 f;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int chunk = (4 * (i & 3) + 2 * dgrp + ((c16 & 3) >> 1)) ^ swz_v<D>(c16 >> 2);
                    const uint8_t *src = vt + (4 * half + (c16 >> 2)) * kRowB + chunk * 16 + (c16 & 1) * 8 + (16 * st + 8 * x) * kRowB + (i >> 2) * 256;
                    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(src));
                    if (x == 0) __builtin_memcpy(&f.x, &v, 8);
                    else __builtin_memcpy(&f.z, &v, 8);
                }
                o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(f), as_bf16x8(p[st]), o[i], 0, 0, 0);
            }
    };
    int spoiled_lo = lk, spoiled_hi = 0;  // keys of the tiles with a find
    auto clear_masked = [&](int key0, uint8_t *vt, const uint32_t (&found)[4]) __attribute__((always_inline)) {
        if (clean(key0)) return;
        if (__builtin_expect(__builtin_amdgcn_readfirstlane(found[0] | found[1] | found[2] | found[3]) == 0, 1)) return;
        spoiled_lo = key0 < spoiled_lo ? key0 : spoiled_lo;
        spoiled_hi = key0 + kKeys < lk ? key0 + kKeys : lk;
#pragma unroll 1
        for (int at = threadIdx.x * 16; at < kTileB; at += 4096) {
            u32x4 w = *reinterpret_cast<const u32x4 *>(vt + at);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if ((w[e] & 0x7F80u) == 0x7F80u) w[e] &= 0xFFFF0000u;
                if ((w[e] & 0x7F800000u) == 0x7F800000u) w[e] &= 0xFFFFu;
            }
            *reinterpret_cast<u32x4 *>(vt + at) = w;
        }
        __syncthreads();
    };

    // The next tile's scores are formed while this tile's weights are: the matrix core and
    // the vector units then work at once within a wave, not only between the two waves of a SIMD.
    if (lo < hi) {
        f32x16 s0[kSub], s1[kSub];
        uint4 p[2 * kSub];
        stage_k(lo, sm_k0);
        load_q();
        __syncthreads();
        if (lo + kKeys < hi) stage_k(lo + kKeys, sm_k1);
        stage_v(lo, sm_v0);
        scores(sm_k0, s0);
        settle(lo, s0, sm_v0, sm_found[0]);
        int key0 = lo;
        // `now`: scores of tile key0; k_next, v_now: the buffers that hold what this pass reads
        auto pass = [&](f32x16 (&now)[kSub], f32x16 (&next)[kSub], uint8_t *k_now, const uint8_t *k_next, uint8_t *v_now,
                        uint8_t *v_next, const uint32_t (&found)[4], uint32_t (&found_next)[4]) __attribute__((always_inline)) {
            __syncthreads();  // K of the next tile and V of this one have arrived; the other buffers are free
            clear_masked(key0, v_now, found);
            if (key0 + 2 * kKeys < hi) stage_k(key0 + 2 * kKeys, k_now);
            stage_v(key0 + kKeys, v_next);
            scores(k_next, next);
            weights(now, p);
            values(v_now, p);
            settle(key0 + kKeys, next, v_next, found_next);
            key0 += kKeys;
        };
        while (key0 + 2 * kKeys < hi) {
            pass(s0, s1, sm_k0, sm_k1, sm_v0, sm_v1, sm_found[0], sm_found[1]);
            pass(s1, s0, sm_k1, sm_k0, sm_v1, sm_v0, sm_found[1], sm_found[0]);
        }
        if (key0 + kKeys < hi) {
            pass(s0, s1, sm_k0, sm_k1, sm_v0, sm_v1, sm_found[0], sm_found[1]);
            __syncthreads();
            clear_masked(key0, sm_v1, sm_found[1]);
            weights(s1, p);
            values(sm_v1, p);
        } else {
            __syncthreads();
            clear_masked(key0, sm_v0, sm_found[0]);
            weights(s0, p);
            values(sm_v0, p);
        }
    }

    // a weight times an infinity or NaN is that again, whatever the weight of a key that is seen
#pragma unroll 1
    for (int key = spoiled_lo; key < spoiled_hi; ++key) {
        if (key < lb || key >= ub) continue;
        const uint16_t *vp = vb + key * a.v_tok + 4 * half;
#pragma unroll
        for (int i = 0; i < kDT; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const u32x2 w = *reinterpret_cast<const u32x2 *>(vp + 32 * i + 8 * x);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
                    o[i][4 * x + e] += __builtin_fabsf(v) < INFINITY ? 0.0f : v;
                }
            }
    }

    l += other_half(l);
    if (!live) return;
    if (range.parts > 1) {
        // unnormalised sums of this part of the keys; k_attn_prefill_join adds the parts
        const int64_t at = ((int64_t)(x * a.kv_heads + hkv) * a.splits + split) * kRows + wave * 32 + col;
        if (half == 0) *reinterpret_cast<float2 *>(a.part_ml + 2 * at) = make_float2(m, l);
        if (lo < hi) {
#pragma unroll
            for (int i = 0; i < kDT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<float4 *>(a.part_o + at * D + 32 * i + 8 * e + 4 * half) =
                        make_float4(o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]);
        }
        return;
    }
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
    if (a.lse && half == 0)
        a.lse[(q0 + tok) * a.heads + head] = (m + __builtin_amdgcn_logf(l)) * 0.69314718f;
    // the lane holds d = 32 i + 8 x + 4 half + (0..3) of its row
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int64_t at = (q0 + tok) * a.o_tok + head * a.o_head + 32 * i + 8 * x + 4 * half;
            const float4 v = make_float4(o[i][4 * x] * f, o[i][4 * x + 1] * f, o[i][4 * x + 2] * f, o[i][4 * x + 3] * f);
            if (a.out_bf16)
                *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(a.out) + at) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
            else
                *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + at) = v;
        }
}

// Adds up the parts of a row tile's keys: 1024 / D rows a workgroup, four d a thread.
template <int D>
__global__ __launch_bounds__(256) void k_attn_prefill_join(PrefillArgs a)
{
    constexpr int kLanes = D / 4, kPer = 256 / kLanes;
    const int xh = blockIdx.x / (kRows / kPer), r = (blockIdx.x - xh * (kRows / kPer)) * kPer + threadIdx.x / kLanes;
    const int x = xh / a.kv_heads, hkv = xh - x * a.kv_heads;
    const QTile qt = find_tile(a, x);
    if (qt.b < 0) return;
    const int64_t q0 = qt.q0, row = (int64_t)qt.tile * kRows + r;
    if (row >= (int64_t)qt.lq * a.group) return;
    const int tok = (int)((uint32_t)row / (uint32_t)a.group), head = hkv * a.group + (int)row - tok * a.group;
    const int parts = key_range<(D == 256 ? 32 : 64)>(a, qt).parts;
    if (parts == 1) return;  // written by its workgroup
    const int64_t first = (int64_t)xh * a.splits * kRows + r;
    float M = -INFINITY;
    for (int s = 0; s < parts; ++s) M = fmaxf(M, a.part_ml[2 * (first + s * kRows)]);
    const float Ms = M == -INFINITY ? 0.0f : M;
    const int d = threadIdx.x % kLanes * 4;
    f32x4 acc = {0, 0, 0, 0};
    float L = 0.0f;
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
        const int64_t at = first + s * kRows;
        const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + 2 * at);
        if (ml.y == 0.0f) continue;  // saw no key; its sums may not have been written
        const float f = __builtin_amdgcn_exp2f(ml.x - Ms);
        L += f * ml.y;
        acc += f * *reinterpret_cast<const f32x4 *>(a.part_o + at * D + d);
    }
    acc *= L == 0.0f ? 0.0f : 1.0f / L;
    const int64_t p = (q0 + tok) * a.o_tok + head * a.o_head + d;
    if (a.out_bf16)
        *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(a.out) + p) = make_uint2(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]));
    else
        *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(a.out) + p) = acc;
    if (a.lse && d == 0) a.lse[(q0 + tok) * a.heads + head] = (M + __builtin_amdgcn_logf(L)) * 0.69314718f;
}

// Row tiles of all sequences and key heads: at most one more per sequence than the packed
// rows hold (of many sequences, empty ones too).
int64_t prefill_grid(int64_t q_tokens, int64_t seqs, int64_t kv_heads, int64_t group)
{
    const int64_t more = seqs < q_tokens || seqs > kManySeqs ? seqs : q_tokens;
    return (q_tokens * group / kRows + more) * kv_heads;
}

// The most parts of a row tile's keys: where the row tiles do not fill half of the workgroups the
// chip holds (two a CU, one at head_dim 256), as many as do, but no more than a row tile has work for
// (key_range).  How long the longest sequence is only the device knows: four times the mean here, which
// keeps a batch of short prompts in one launch (16 of 64 tokens 16.6 -> 12.4 us, 16 of 200 22.3 -> 12.3) and
// a long one among short ones split (3000 tokens beside seven of 2 to 600: 43.5 us, by twice the mean 54.1).
int prefill_splits(int64_t q_tokens, int64_t k_tokens, int64_t seqs, int64_t kv_heads, int64_t group, int64_t head_dim,
                   int64_t window)
{
    const int64_t grid = prefill_grid(q_tokens, seqs, kv_heads, group);
    const int64_t room = device_cu_count() * (head_dim == 256 ? 1 : 2) / (grid > 0 ? grid : 1);
    const int64_t mean = (k_tokens + seqs - 1) / seqs;
    int64_t keys = 4 * mean < k_tokens ? 4 * mean : k_tokens;
    if (window > 0 && window < keys - 2 * kRows) keys = window + 2 * kRows;  // a row tile's tokens, to whole tiles of keys
    const int64_t most = keys / kPartKeys;
    const int64_t s = room < most ? room : most;
    return s < 1 ? 1 : (s > 64 ? 64 : (int)s);
}

size_t prefill_part_rows(int64_t q_tokens, int64_t seqs, int64_t kv_heads, int64_t group, int splits)
{
    return splits > 1 ? (size_t)(prefill_grid(q_tokens, seqs, kv_heads, group) * splits * kRows) : 0;
}

template <int D>
static fp4_status launch_d(const PrefillArgs &a, int64_t grid, hipStream_t st)
{
    // a launch holds less than 2^32 threads (only calls without splits come near)
    const int64_t blocks = grid * a.splits, most = int64_t(1) << 23;
    for (int64_t first = 0; first < blocks; first += most) {
        PrefillArgs part = a;
        part.first = (int)first;
        hipLaunchKernelGGL(k_attn_prefill<D>, dim3((unsigned)(blocks - first < most ? blocks - first : most)), dim3(256), 0, st, part);
    }
    if (a.splits > 1)
        hipLaunchKernelGGL(k_attn_prefill_join<D>, dim3((unsigned)(grid * (kRows * D / 1024))), dim3(256), 0, st, a);
    return hipGetLastError() == hipSuccess ? FP4_OK : FP4_ERR_HIP;
}

fp4_status launch_attn_prefill(const PrefillArgs &a, hipStream_t st)
{
    const int64_t grid = prefill_grid(a.q_tokens, a.seqs, a.kv_heads, a.group);
    PrefillArgs f = a;
    const int cus = device_cu_count();
    f.fold_at = (cus + a.kv_heads - 1) / a.kv_heads;  // row tiles that come one to a CU
    f.fold_most = a.splits == 1 && a.head_dim < 256 ? 2 * cus : 0;
    if (a.head_dim == 64) return launch_d<64>(f, grid, st);
    if (a.head_dim == 128) return launch_d<128>(f, grid, st);
    return launch_d<256>(f, grid, st);
}

}  // namespace fp4k
