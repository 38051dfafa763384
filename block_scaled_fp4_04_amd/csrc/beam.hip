// beam.hip -- beam search's selection: of every group of beams the k best continuations over beams and
// vocabulary.
//
//   total(i, v) = score_i + logit_iv - log sum_u exp(logit_iu)
//
// Two launches.  k_beam_rows reads the logits once, a workgroup a part of a row: the part's maximum, its sum of
// exponentials and its k best logits (within a row the order of the totals is that of the logits).  k_beam_join
// adds up a row's sums, and merges the sorted lists of all parts of all beams.  Bound by reading the logits, and then by
// what follows the last load: 461 rows of 131072 bf16 logits (121 MB) take 30 us (24 us without exponentials and
// selection, 19 us is the time of a load-only pass) and the join of 64 groups, k = 16, 6.8 us.
//
// Order: totals are compared in 64 bits (in 32, sums of scores around -50 and small differences of logits
// would merge neighbours), equal ones by beam, logit and token: beside a score of -10^30, or a maximum 10^17 times as
// large, 64 bits hold no difference of logits either, and a beam's list has to be as sorted by totals as it is by logits.
//
// The sums of exponentials are fp32 over a lane's values of a group (32 or 16, by halves) and 64 bits from there on.  The
// exponentials are fp32, e^a of a = logit - reference: v_exp_f32
// is within 1 ulp, and a's two roundings and that of log2 e weigh 1.2 |a| 2^-23 at most.  The reference is a wave's first
// maximum until a value is more than 8 above it, so a term d below the row's maximum has |a| <= max(8, d), and the mean of that
// over a row's N terms, each weighed by its share, is at most max(9, ln N) (entropy).  The additions and the exponentials
// that match two references are 5 ulp at most.  So a row's sum is within (7 + 1.2 max(9, ln N)) 2^-23 of itself: less than
// 2^-18 for any row, and about 2^-25 in practice, as the errors have either sign.
#include "device_common.h"
#include "internal.h"

namespace fp4k {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

template <typename T>
struct Row;

template <>
struct Row<uint16_t> {
    static constexpr int kPer = 8, kKeyShift = 16;  // bf16: 16 bits of the key tell all values apart
    static constexpr uint32_t kNone = 0xFF80FF80u;  // -infinity
    static __device__ __forceinline__ void put(uint32_t (&w)[4], int j, uint16_t v)
    {
        w[j >> 1] = (j & 1) ? (w[j >> 1] & 0xFFFFu) | ((uint32_t)v << 16) : (w[j >> 1] & 0xFFFF0000u) | v;
    }
    static __device__ __forceinline__ float get(const uint32_t (&w)[4], int j)
    {
        return __uint_as_float((j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
    }
};

template <>
struct Row<float> {
    static constexpr int kPer = 4, kKeyShift = 0;
    static constexpr uint32_t kNone = 0xFF800000u;
    static __device__ __forceinline__ void put(uint32_t (&w)[4], int j, float v) { w[j] = __float_as_uint(v); }
    static __device__ __forceinline__ float get(const uint32_t (&w)[4], int j) { return __uint_as_float(w[j]); }
};

// fp32 bits in an order that unsigned numbers have, and back
__device__ __forceinline__ uint32_t order_of(float f)
{
    const uint32_t u = __float_as_uint(f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : ~0u)); }

template <int CTRL>
__device__ __forceinline__ int dpp(int v)
{
    return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, false);
}

// lane ^ M's value; within a row of 16 lanes by DPP
template <int M>
__device__ __forceinline__ int lane_xor(int v)
{
    if constexpr (M == 1) return dpp<0xB1>(v);
    else if constexpr (M == 2) return dpp<0x4E>(v);
    else if constexpr (M == 3) return dpp<0x1B>(v);
    else if constexpr (M == 7) return dpp<0x141>(v);   // half mirror
    else if constexpr (M == 4) return dpp<0x1B>(dpp<0x141>(v));
    else if constexpr (M == 15) return dpp<0x140>(v);  // mirror
    else if constexpr (M == 8) return dpp<0x128>(v);   // rotation by 8 of 16
    else return __shfl_xor(v, M, kWave);
}

// lane i takes lane i - 1's value
__device__ __forceinline__ int wave_shr1(int v) { return __builtin_amdgcn_mov_dpp(v, 0x138, 0xF, 0xF, false); }

constexpr int kVec = 4;      // 16-byte vectors of a lane in a group
constexpr int kMost = 8;     // groups of a part, at most
constexpr int kListed = 64;  // vectors listed before they are looked through

// The k best of a wave so far, best first, in lanes 0 .. k - 1
struct Best {
    float v;
    int i;
};

// val (uniform) into its place, if it has one: behind what is equal, which came before it
__device__ __forceinline__ void insert(Best &s, float val, int idx, uint64_t seats, int lane)
{
    const uint64_t beaten = __ballot(val > s.v) & seats;
    if (!beaten) return;
    const int at = __builtin_ctzll(beaten);
    const float pv = __int_as_float(wave_shr1(__float_as_int(s.v)));
    const int pi = wave_shr1(s.i);
    s.v = lane > at ? pv : lane == at ? val : s.v;
    s.i = lane > at ? pi : lane == at ? idx : s.i;
}

__device__ __forceinline__ float lane_of(float v, int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane)); }

// Maximum and sum over a wave, the same in every lane: within rows of 16 lanes by DPP, then the four rows'
__device__ __forceinline__ float wave_top(float v)
{
    v = fmaxf(v, __int_as_float(lane_xor<1>(__float_as_int(v))));
    v = fmaxf(v, __int_as_float(lane_xor<2>(__float_as_int(v))));
    v = fmaxf(v, __int_as_float(lane_xor<7>(__float_as_int(v))));
    v = fmaxf(v, __int_as_float(lane_xor<15>(__float_as_int(v))));
    return fmaxf(fmaxf(lane_of(v, 0), lane_of(v, 16)), fmaxf(lane_of(v, 32), lane_of(v, 48)));
}

// e^d, d <= 0, by v_exp_f32 of what is left of a whole power of two: the rounding of that argument does not grow with d
__device__ __forceinline__ double exp_of(double d)
{
    const double x = fmax(d * 1.4426950408889634, -2000.0), n = __builtin_rint(x);
    return __builtin_amdgcn_ldexp((double)__builtin_amdgcn_exp2f((float)(x - n)), (int)n);
}

template <typename V, typename Get>
__device__ __forceinline__ V moved(V v, Get get)
{
    static_assert(sizeof(V) == 8, "two words");
    uint64_t u;
    __builtin_memcpy(&u, &v, 8);
    u = ((uint64_t)(uint32_t)get((int)(u >> 32)) << 32) | (uint32_t)get((int)u);
    __builtin_memcpy(&v, &u, 8);
    return v;
}

__device__ __forceinline__ double wave_sum(double v)
{
    v += moved(v, [](int x) { return lane_xor<1>(x); });
    v += moved(v, [](int x) { return lane_xor<2>(x); });
    v += moved(v, [](int x) { return lane_xor<7>(x); });
    v += moved(v, [](int x) { return lane_xor<15>(x); });
    auto row = [&](int r) { return moved(v, [r](int x) { return __builtin_amdgcn_readlane(x, r); }); };
    return (row(0) + row(16)) + (row(32) + row(48));
}

// Sorted runs of KP lanes, best first.  Best: a value of a row; Entry: a total of a group.

struct Entry {
    double total;
    uint64_t place;  // beam, the logit's order from above, token; kNowhere: none
};
constexpr uint64_t kNowhere = ~0ull;  // (beams * vocab <= 2^30: beam and token take 31 bits at most)

__device__ __forceinline__ bool better(const Best &x, const Best &y) { return x.v > y.v || (x.v == y.v && x.i < y.i); }
__device__ __forceinline__ bool better(const Entry &x, const Entry &y)
{
    return x.total > y.total || (x.total == y.total && x.place < y.place);
}

template <int M>
__device__ __forceinline__ Best lane_xor(const Best &x)
{
    return Best{__int_as_float(lane_xor<M>(__float_as_int(x.v))), lane_xor<M>(x.i)};
}
template <int M>
__device__ __forceinline__ Entry lane_xor(const Entry &x)
{
    auto get = [](int v) { return lane_xor<M>(v); };
    return Entry{moved(x.total, get), moved(x.place, get)};
}

// x: a bitonic run of 2 D lanes -> sorted, best first
template <int D, typename E>
__device__ __forceinline__ void settle(E &x, int lane)
{
    const E y = lane_xor<D>(x);
    if ((lane & D) ? better(x, y) : better(y, x)) x = y;
    if constexpr (D > 1) settle<D / 2>(x, lane);
}

// Sorted runs x and y of KP lanes: the best of both, sorted.  Against the reverse of y, the better of each
// pair are the KP best, and form a bitonic run.
template <int KP, typename E>
__device__ __forceinline__ void merge(E &x, const E &y, int lane)
{
    const E z = lane_xor<KP - 1>(y);
    if (better(z, x)) x = z;
    settle<KP / 2>(x, lane);
}

// all runs of a wave into one (every run ends up as it), H lanes of them done
template <int KP, int H, typename E>
__device__ __forceinline__ void merge_wave(E &x, int lane)
{
    if constexpr (H < 64) {
        const E z = lane_xor<(H | (KP - 1))>(x);
        if (better(z, x)) x = z;
        settle<KP / 2>(x, lane);
        merge_wave<KP, 2 * H>(x, lane);
    }
}

// A group of vectors from token e0 on.  Vectors begin at multiples of kPer tokens whatever the row's address
// (unaligned 16-byte loads), so that equal rows have equal sums and their ties go to the lowest beam.
template <bool ONCE, typename T>
__device__ __forceinline__ void load_group(uint32_t (&w)[kVec][4], const T *x, int e0, int vocab, int lane)
{
    typedef u32x4 vec __attribute__((aligned(2)));
    constexpr int kPer = Row<T>::kPer;
    int e = e0 + lane * kPer;
    if (e0 + kVec * 64 * kPer <= vocab) {
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            const vec *p = reinterpret_cast<const vec *>(x + e + v * 64 * kPer);
            const u32x4 r = ONCE ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
            for (int c = 0; c < 4; ++c) w[v][c] = r[c];
        }
        return;
    }
#pragma unroll
    for (int v = 0; v < kVec; ++v, e += 64 * kPer) {
        if (e + kPer <= vocab) {
            __builtin_memcpy(w[v], x + e, 16);
        } else {
            w[v][0] = w[v][1] = w[v][2] = w[v][3] = Row<T>::kNone;
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (e + j < vocab) Row<T>::put(w[v], j, x[e + j]);
        }
    }
}

template <typename T>
__device__ __forceinline__ float widen(T v)
{
    if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)v << 16);
    else return v;
}

// A workgroup takes a part of a row, each of its W waves a.groups groups one behind the other, the next group's loads in
// flight; with four waves one of them then adds up the four sums and merges the four lists.
//
// First pass: sums of exponentials, and every vector's maximum into LDS.  The k-th largest of the lanes'
// maxima is then a bar that at least k values reach and all of the k best do.  Second pass: the vectors whose
// maximum reaches it (about k of them) are listed and read again, and their values put in their places one at a
// time, the bar rising.
template <typename T, int KP, int W, bool ONCE>
__global__ __launch_bounds__(64 * W) void k_beam_rows(BeamArgs a)
{
    constexpr int kPer = Row<T>::kPer, kGroup = kVec * 64 * kPer;
    constexpr float kLowest = -3.4028234663852886e38f;
    const float kInf = __builtin_inff();
    __shared__ float4 sm_top[W][kMost][64];
    __shared__ int sm_listed[W][kListed + kVec * 64];
    __shared__ float sm_ref[W];
    __shared__ double sm_sum[W];
    __shared__ Best sm_best[W][KP];
    const int wave = W > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0, lane = threadIdx.x & 63;
    const int64_t id = blockIdx.x;
    const int row = (int)(id / a.parts), part = (int)(id - (int64_t)row * a.parts);
    if (a.done && a.done[row]) return;
    const T *x = reinterpret_cast<const T *>(a.logits) + row * a.ld;
    const int first = (part * W + wave) * a.groups * kGroup;
    const int groups = min(a.groups, (a.vocab - first + kGroup - 1) / kGroup);  // (<= 0 past the row's end)
    uint32_t w[kVec][4];
    load_group<ONCE>(w, x, first, a.vocab, lane);

    // Exponentials are taken against the first group's maximum `ref` until a value is more than 8 above it (rounding, above).
    // (2^(x log2e - c) is one instruction less a value, but then a term at the reference is not exact.)
    float top = -kInf;  // NaN is passed over here and spoils the sum
#pragma unroll
    for (int v = 0; v < kVec; ++v)
#pragma unroll
        for (int j = 0; j < kPer; ++j) top = fmaxf(top, Row<T>::get(w[v], j));
    float ref = fmaxf(wave_top(top), kLowest);
    double sum = 0.0;
    for (int g = 0; g < groups; ++g) {
        uint32_t next[kVec][4];
        if (g + 1 < groups) load_group<ONCE>(next, x, first + (g + 1) * kGroup, a.vocab, lane);
        float m[kVec];
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            m[v] = -kInf;
#pragma unroll
            for (int j = 0; j < kPer; ++j) m[v] = fmaxf(m[v], Row<T>::get(w[v], j));
        }
        sm_top[wave][g][lane] = make_float4(m[0], m[1], m[2], m[3]);
        const float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
        top = fmaxf(top, most);
        if (__ballot(most - ref > 8.0f)) {
            const float now = wave_top(most);
            sum *= exp((double)ref - (double)now);
            ref = now;
        }
        float part_sum = 0.0f;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            float f[kPer];
#pragma unroll
            for (int j = 0; j < kPer; ++j) f[j] = __builtin_amdgcn_exp2f((Row<T>::get(w[v], j) - ref) * kLog2e);
#pragma unroll
            for (int d = kPer / 2; d > 0; d >>= 1)
#pragma unroll
                for (int j = 0; j < d; ++j) f[j] += f[j + d];
            part_sum += f[0];
        }
        sum += (double)part_sum;
#pragma unroll
        for (int v = 0; v < kVec; ++v)
#pragma unroll
            for (int c = 0; c < 4; ++c) w[v][c] = next[v][c];
    }
    sum = wave_sum(sum);
    if (W > 1 && lane == 0) {
        sm_ref[wave] = ref;
        sm_sum[wave] = sum;
    }

    // the bar, bit by bit from the top, by counting lanes; what counts is above it
    const uint32_t key = order_of(top) >> Row<T>::kKeyShift;
    uint32_t t = 0;
    for (int b = 31 - Row<T>::kKeyShift; b >= 0; --b) {
        const uint32_t c = t | (1u << b);
        if (__builtin_popcountll(__ballot(key >= c)) >= a.k) t = c;
    }
    float bar = __uint_as_float(__float_as_uint(value_of(t << Row<T>::kKeyShift)) & (~0u << Row<T>::kKeyShift));
    if (bar > -kInf) bar = bar == 0.0f ? -0x1p-149f : value_of(order_of(bar) - 1);

    Best s{-kInf, 0x7FFFFFFF};
    const uint64_t seats = ~0ull >> (64 - a.k);
    int *listed = sm_listed[wave], n = 0;
    // the listed vectors, 64 / kPer at a time, a value a lane, in the order of the tokens; four such loads in flight
    auto look = [&]() {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        constexpr int kOnce = 64 / kPer;
        for (int i0 = 0; i0 < n; i0 += 4 * kOnce) {
            float f[4];
            int at[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int i = i0 + c * kOnce + lane / kPer;
                at[c] = i < n ? listed[i] + lane % kPer : a.vocab;
                f[c] = at[c] < a.vocab ? widen(x[at[c]]) : -kInf;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
                for (uint64_t in = __ballot(f[c] > bar); in; in &= in - 1) {
                    const int l = __builtin_ctzll(in);
                    insert(s, lane_of(f[c], l), __builtin_amdgcn_readlane(at[c], l), seats, lane);
                    bar = fmaxf(bar, lane_of(s.v, a.k - 1));
                }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        n = 0;
    };
    for (int g = 0; g < groups; ++g) {
        const float4 q = sm_top[wave][g][lane];
        const float m[kVec] = {q.x, q.y, q.z, q.w};
        uint64_t hit[kVec];
#pragma unroll
        for (int v = 0; v < kVec; ++v) hit[v] = __ballot(m[v] > bar);
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            if (!hit[v]) continue;
            if ((hit[v] >> lane) & 1ull)
                listed[n + __builtin_popcountll(hit[v] & ((1ull << lane) - 1))] = first + g * kGroup + (v * 64 + lane) * kPer;
            n += __builtin_popcountll(hit[v]);
        }
        if (n >= kListed) look();
    }
    look();
    Best best = s;
    if constexpr (W > 1) {
        static_assert(W == 4, "four lists are merged");
        if (lane < KP) sm_best[wave][lane] = s;  // (lanes from k on hold what was displaced, in order)
        __syncthreads();
        if (wave > 0) return;
        constexpr int kRuns = 64 / KP < W ? 64 / KP : W;
        const int run = lane / KP;
        best = run < W ? sm_best[run < W ? run : 0][lane % KP] : Best{-kInf, 0x7FFFFFFF};
#pragma unroll
        for (int r = kRuns; r < W; r += kRuns) merge<KP>(best, sm_best[r + run][lane % KP], lane);
        merge_wave<KP, KP>(best, lane);
        ref = fmaxf(fmaxf(sm_ref[0], sm_ref[1]), fmaxf(sm_ref[2], sm_ref[3]));
        sum = 0.0;
#pragma unroll
        for (int r = 0; r < W; ++r) sum += sm_sum[r] * exp_of((double)sm_ref[r] - (double)ref);
    }
    if (lane < a.k) {
        a.part_value[id * a.k + lane] = best.v;
        a.part_token[id * a.k + lane] = best.i;
    }
    if (lane == 0) {
        a.part_top[id] = ref;
        a.part_sum[id] = sum;
    }
}

// ---------------------------------------------------------------- join --

// One workgroup a group of beams; lists of KP places, a.k of them in use
template <int KP>
__global__ __launch_bounds__(1024) void k_beam_join(BeamArgs a)
{
    __shared__ double base[64];  // score - log of the sum against ...
    __shared__ float from[64];   // ... this logit
    __shared__ Entry found[16][KP];
    const double kInf = __builtin_inf();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int row0 = (int)blockIdx.x * a.beams;
    constexpr int kPer = 64 / KP;
    const int lists = a.beams * a.parts, slot = lane & (KP - 1);

    // One list place; of an ended beam the first one stands for its own score (+0).  What an ended beam's rows
    // hold in the workspace is old, and not used.  All loads are issued before any is waited for, here and
    // below: the data comes from the other chiplets' caches, and a wait costs more than the arithmetic.
    auto load = [&](int l, float &v, uint32_t &token, int &beam) {
        const bool is = l < lists && slot < a.k;
        beam = is ? l / a.parts : 0;
        const int64_t at = is ? ((int64_t)row0 * a.parts + l) * a.k + slot : 0;
        const uint8_t ended = a.done ? a.done[row0 + beam] : 0;
        v = a.part_value[at];
        token = (uint32_t)a.part_token[at];
        if (ended) {
            v = l == beam * a.parts && slot == 0 ? 0.0f : -__builtin_inff();
            token = (uint32_t)a.end_token;
        }
        if (!is) v = -__builtin_inff();
    };
    float v;
    uint32_t token;
    int beam;
    load(wave * kPer + lane / KP, v, token, beam);

    // score - log of the whole row's sum; an ended beam's score
    for (int i = wave; i < a.beams; i += waves) {
        const int row = row0 + i;
        const int64_t at = (int64_t)row * a.parts;
        const uint8_t ended = a.done ? a.done[row] : 0;
        const double b = (double)a.scores[row];
        float top = -__builtin_inff();
        double sum = 0.0;
        for (int p0 = 0; p0 < a.parts; p0 += 64) {
            const int p = p0 + lane;
            const float t = p < a.parts ? a.part_top[at + p] : -__builtin_inff();
            const double u = p < a.parts ? a.part_sum[at + p] : 0.0;
            const float now = fmaxf(top, wave_top(t));
            if (p0 > 0 && now > top) sum *= exp((double)top - (double)now);
            sum += p < a.parts ? u * exp_of((double)t - (double)now) : 0.0;
            top = now;
        }
        const double rest = log(wave_sum(sum));
        if (lane == 0) {
            base[i] = ended ? b : b - rest;
            from[i] = ended ? 0.0f : top;
        }
    }
    __syncthreads();

    const int token_bits = 32 - __builtin_clz((a.vocab - 1) | 1);
    Entry best{-kInf, kNowhere};
    for (int l0 = wave * kPer; l0 < lists; l0 += waves * kPer) {
        if (l0 != wave * kPer) load(l0 + lane / KP, v, token, beam);
        Entry e{-kInf, kNowhere};
        if (v > -__builtin_inff()) {
            const double total = ((double)v - (double)from[beam]) + base[beam];
            const uint32_t below = ~order_of(v + 0.0f);  // (-0 and 0 are equal)
            if (total > -kInf) e = Entry{total, ((((uint64_t)beam << 32) | below) << token_bits) | token};  // (NaN is not)
        }
        if (l0 == wave * kPer) best = e;
        else merge<KP>(best, e, lane);
    }
    merge_wave<KP, KP>(best, lane);
    if (waves > 1) {
        if (lane < KP) found[wave][lane] = best;
        __syncthreads();
        if (wave > 0) return;
        for (int w = lane / KP; w - lane / KP < waves; w += kPer) {
            const Entry e = w < waves ? found[w][slot] : Entry{-kInf, kNowhere};
            if (w < kPer) best = e;
            else merge<KP>(best, e, lane);
        }
        merge_wave<KP, KP>(best, lane);
    }
    // Fewer totals above -infinity than places: all of them are chosen, and the others follow in the order of beam and
    // token, that is the n-th number that is not among the chosen ones: x = n + how many of them are <= x.
    const bool is_real = best.place != kNowhere;
    const int real = __builtin_popcountll(__ballot(lane < a.k && is_real));
    uint32_t parent = (uint32_t)(best.place >> (32 + token_bits));
    token = (uint32_t)best.place & ((1u << token_bits) - 1u);
    if (real < a.k) {
        const uint32_t n = (uint32_t)(lane - real), flat = parent * (uint32_t)a.vocab + token;
        uint32_t x = n;
        for (bool more = true; more;) {
            uint32_t y = n;
            for (int i = 0; i < real; ++i) y += (uint32_t)__builtin_amdgcn_readlane((int)flat, i) <= x;
            more = __ballot(lane >= real && y != x) != 0;
            x = y;
        }
        if (lane >= real) {
            best.total = -kInf;
            parent = x / (uint32_t)a.vocab;
            token = x - parent * (uint32_t)a.vocab;
        }
    }
    if (lane < a.k) {
        const int64_t at = (int64_t)blockIdx.x * a.k + lane;
        a.out_scores[at] = (float)best.total;
        a.out_parents[at] = (int32_t)parent;
        a.out_tokens[at] = (int32_t)token;
    }
}

template <typename T, int KP>
void launch_kp(const BeamArgs &a, const BeamShape &shape, hipStream_t st)
{
    const dim3 grid((unsigned)((int64_t)a.batch * a.beams * a.parts));
    // Logits past the caches' size are read with the non-temporal hint (512 rows of 131072 in bf16, 134 MB: k = 4 36.3 -> 33.7
    // us a call, k = 16 38.7 -> 37.5, behind the product that makes them 287.7 -> 285.8 together; 34 MB and less 0.2 to 1 us
    // slower with it, when they have been read shortly before)
    const bool once = (int64_t)a.batch * a.beams * a.vocab * (int64_t)sizeof(T) >= (int64_t(96) << 20);
    if (shape.waves == 1) {
        if (once) hipLaunchKernelGGL((k_beam_rows<T, KP, 1, true>), grid, dim3(64), 0, st, a);
        else hipLaunchKernelGGL((k_beam_rows<T, KP, 1, false>), grid, dim3(64), 0, st, a);
    } else {
        if (once) hipLaunchKernelGGL((k_beam_rows<T, KP, 4, true>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_beam_rows<T, KP, 4, false>), grid, dim3(256), 0, st, a);
    }
    // a wave a list step and a beam, up to 8, or 16 where there are very many lists
    const int64_t lists = (int64_t)a.beams * a.parts, steps = (lists + 64 / KP - 1) / (64 / KP), most = steps > a.beams ? steps : a.beams;
    const int cap = steps > 128 ? 16 : 8;
    int waves = 1;
    while (waves < most && waves < cap) waves <<= 1;
    hipLaunchKernelGGL(k_beam_join<KP>, dim3((unsigned)a.batch), dim3(64 * waves), 0, st, a);
}

template <typename T>
void launch_k(const BeamArgs &a, const BeamShape &shape, hipStream_t st)
{
    if (a.k <= 4) launch_kp<T, 4>(a, shape, st);
    else if (a.k <= 8) launch_kp<T, 8>(a, shape, st);
    else if (a.k <= 16) launch_kp<T, 16>(a, shape, st);
    else if (a.k <= 32) launch_kp<T, 32>(a, shape, st);
    else launch_kp<T, 64>(a, shape, st);
}

}  // namespace

// Groups of a wave: as many as leave the chip a wave a SIMD (fewer lists to join; 4 / 2 / 1 waves a SIMD: 16 groups of 8
// beams of 131072 tokens 21.3 / 19.5 / 19.1 us, 32 of 5 of 50003 19.9 / 20.0 / 16.2 us, the others alike).
// Waves of a workgroup: one where its lists are few enough for one step of the join's 8 waves, else four, which merge
// theirs (one / four, us a call: 4 beams of 32000, k = 4, 10.1 / 11.6; 64 batches of it 13.5 / 15.1; 512 of 8 beams, k = 16,
// 66.1 / 81.9; 4096 of 4 beams of 4000 tokens 66.6 / 147; past that step, 64 of 8 beams of 131072, k = 16, 39.1 / 37.5).
BeamShape beam_shape(int64_t rows, int64_t beams, int64_t vocab, int64_t k, fp4_dtype xt)
{
    const int64_t group = kVec * 64 * (xt == FP4_BF16 ? 8 : 4);
    const int64_t all = rows * ((vocab + group - 1) / group) / (4 * device_cu_count());
    BeamShape s;
    s.groups = all < 1 ? 1 : all > kMost ? kMost : (int)all;
    int64_t kp = 4;  // places of a list (launch_k)
    while (kp < k) kp <<= 1;
    const int64_t alone = (vocab + group * s.groups - 1) / (group * s.groups);
    s.waves = beams * alone * kp <= 8 * 64 ? 1 : 4;
    s.parts = s.waves == 1 ? alone : (vocab + 4 * group * s.groups - 1) / (4 * group * s.groups);
    return s;
}

fp4_status launch_beam_select(BeamArgs a, fp4_dtype xt, hipStream_t st)
{
    const BeamShape shape = beam_shape((int64_t)a.batch * a.beams, a.beams, a.vocab, a.k, xt);
    a.parts = (int)shape.parts;
    a.groups = shape.groups;
    if (xt == FP4_BF16) launch_k<uint16_t>(a, shape, st);
    else launch_k<float>(a, shape, st);
    return hipGetLastError() == hipSuccess ? FP4_OK : FP4_ERR_HIP;
}

}  // namespace fp4k
