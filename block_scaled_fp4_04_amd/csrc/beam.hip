// beam.hip -- beam search's selection: of every group of beams the k best continuations over beams and
// vocabulary.
//
//   total(i, v) = score_i + logit_iv - log sum_u exp(logit_iu)
//
// Two launches.  k_beam_rows reads every logit once: a wave takes a part of a row into registers, forms the
// part's maximum and its sum of exponentials, and its k best logits (within a row the order of the totals
// is that of the logits).  k_beam_join adds up a row's sums, and merges the sorted lists of all parts of
// all beams.  Bound by reading the logits.
//
// Order: totals are compared in 64 bits (in 32, sums of scores around -50 and small differences of logits
// would merge neighbours), equal ones by beam * vocab + token.  The sums of exponentials are fp32 over 8
// neighbours and 64 bits from there on; the exponentials are fp32 (v_exp_f32, 1 ulp).
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

// lane i takes lane i - 1's value
__device__ __forceinline__ int wave_shr1(int v) { return __builtin_amdgcn_mov_dpp(v, 0x138, 0xF, 0xF, false); }

// A part of a row: 64 lanes x NV vectors of 16 bytes.
template <typename T, int NV>
__global__ __launch_bounds__(256) void k_beam_rows(BeamArgs a)
{
    constexpr int kPer = Row<T>::kPer;
    const float kInf = __builtin_inff();
    const int64_t id = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (id >= (int64_t)a.batch * a.beams * a.parts) return;
    const int row = (int)(id / a.parts), part = (int)(id - (int64_t)row * a.parts), lane = threadIdx.x & 63;
    if (a.done && a.done[row]) return;
    const T *x = reinterpret_cast<const T *>(a.logits) + row * a.ld;
    // Vectors begin at multiples of kPer tokens whatever the row's address (unaligned 16-byte loads): so
    // equal rows have equal sums, and their ties go to the lowest beam.
    const int first = part * (64 * NV * kPer);
    uint32_t w[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = first + (v * 64 + lane) * kPer;
        if (e + kPer <= a.vocab) {
            __builtin_memcpy(w[v], x + e, 16);
        } else {
            w[v][0] = w[v][1] = w[v][2] = w[v][3] = Row<T>::kNone;
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (e + j < a.vocab) Row<T>::put(w[v], j, x[e + j]);
        }
    }

    // maxima: of each vector, the lane, the part.  NaN is passed over here and spoils the sum below.
    float vmax[NV], lmax = -kInf;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float m = -kInf;
#pragma unroll
        for (int j = 0; j < kPer; ++j) m = fmaxf(m, Row<T>::get(w[v], j));
        vmax[v] = m;
        lmax = fmaxf(lmax, m);
    }
    float top = lmax;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));

    // sum of exponentials against the part's maximum
    const float ref = top == -kInf ? 0.0f : top;
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float e[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) e[j] = __builtin_amdgcn_exp2f((Row<T>::get(w[v], j) - ref) * kLog2e);
#pragma unroll
        for (int d = kPer / 2; d > 0; d >>= 1)
#pragma unroll
            for (int j = 0; j < d; ++j) e[j] += e[j + d];
        sum += (double)e[0];
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, kWave);
    if (lane == 0) {
        a.part_top[id] = top;
        a.part_sum[id] = sum;
    }

    // The k-th largest of the lanes' maxima: at least k values reach it, and no smaller one is among the
    // k best.  Found bit by bit from the top, by counting lanes.
    const uint32_t key = order_of(lmax) >> Row<T>::kKeyShift;
    uint32_t t = 0;
    for (int b = 31 - Row<T>::kKeyShift; b >= 0; --b) {
        const uint32_t c = t | (1u << b);
        if (__builtin_popcountll(__ballot(key >= c)) >= a.k) t = c;
    }
    const float bar = __uint_as_float(__float_as_uint(value_of(t << Row<T>::kKeyShift)) & (~0u << Row<T>::kKeyShift));

    // the k best in lanes 0 .. k - 1, best first: what reaches the bar is put in its place, one at a time
    float lv = -kInf;
    int li = 0x7FFFFFFF;
    const uint64_t seats = ~0ull >> (64 - a.k);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (!__ballot(vmax[v] >= bar && vmax[v] > -kInf)) continue;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const float f = Row<T>::get(w[v], j);
            uint64_t hit = __ballot(f >= bar && f > -kInf);
            while (hit) {
                const int l = __builtin_ctzll(hit);
                hit &= hit - 1;
                const float val = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), l));
                const int idx = first + (v * 64 + l) * kPer + j;
                const uint64_t beaten = __ballot(val > lv || (val == lv && idx < li)) & seats;
                if (!beaten) continue;
                const int at = __builtin_ctzll(beaten);
                const float pv = __int_as_float(wave_shr1(__float_as_int(lv)));
                const int pi = wave_shr1(li);
                lv = lane > at ? pv : lane == at ? val : lv;
                li = lane > at ? pi : lane == at ? idx : li;
            }
        }
    }
    if (lane < a.k) {
        a.part_value[id * a.k + lane] = lv;
        a.part_token[id * a.k + lane] = li;
    }
}

// ---------------------------------------------------------------- join --

struct Entry {
    double total;
    uint32_t flat;  // beam * vocab + token
};

__device__ __forceinline__ bool better(const Entry &x, const Entry &y)
{
    return x.total > y.total || (x.total == y.total && x.flat < y.flat);
}

__device__ __forceinline__ Entry lane_xor(const Entry &x, int mask)
{
    return Entry{__shfl_xor(x.total, mask, kWave), (uint32_t)__shfl_xor((int)x.flat, mask, kWave)};
}

// x: a bitonic run of `kp` lanes -> sorted, best first
__device__ __forceinline__ Entry settle(Entry x, int kp, int lane)
{
    for (int d = kp >> 1; d > 0; d >>= 1) {
        const Entry y = lane_xor(x, d);
        const bool swap = (lane & d) ? better(x, y) : better(y, x);
        if (swap) x = y;
    }
    return x;
}

// sorted runs x and y (the same lanes): the best of both, sorted.  Against the reverse of y, the better of
// each pair are the kp best, and form a bitonic run.
__device__ __forceinline__ Entry merge(Entry x, const Entry &y, int kp, int lane)
{
    const Entry z = lane_xor(y, kp - 1);
    if (better(z, x)) x = z;
    return settle(x, kp, lane);
}

// all runs of a wave into the one of lanes 0 .. kp - 1 (every run ends up the same)
__device__ __forceinline__ Entry merge_wave(Entry x, int kp, int lane)
{
    for (int h = kp; h < 64; h <<= 1) {
        const Entry z = lane_xor(x, h | (kp - 1));
        if (better(z, x)) x = z;
        x = settle(x, kp, lane);
    }
    return x;
}

// One workgroup a group of beams
__global__ __launch_bounds__(1024) void k_beam_join(BeamArgs a, int kp)
{
    __shared__ double base[64];
    __shared__ double sm_total[16 * 64];
    __shared__ uint32_t sm_flat[16 * 64];
    const double kInf = __builtin_inf();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int row0 = (int)blockIdx.x * a.beams;
    // score - log of the whole row's sum
    for (int i = wave; i < a.beams; i += waves) {
        const int row = row0 + i;
        double b = (double)a.scores[row];
        if (!(a.done && a.done[row])) {
            float top = -__builtin_inff();
            for (int p = lane; p < a.parts; p += 64) top = fmaxf(top, a.part_top[(int64_t)row * a.parts + p]);
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
            double sum = 0.0;
            for (int p = lane; p < a.parts; p += 64) {
                const float t = a.part_top[(int64_t)row * a.parts + p];
                const double s = a.part_sum[(int64_t)row * a.parts + p];
                sum += t == -__builtin_inff() ? s : s * exp((double)t - (double)top);
            }
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, kWave);
            b -= (double)top + log(sum);
        }
        if (lane == 0) base[i] = b;
    }
    __syncthreads();

    // lists of kp (k of them real), 64 / kp of them a wave and step
    const int lists = a.beams * a.parts, per = 64 / kp, slot = lane & (kp - 1);
    Entry best{-kInf, ~0u};
    for (int l0 = wave * per; l0 < lists; l0 += waves * per) {
        const int l = l0 + lane / kp;
        Entry e{-kInf, ~0u};
        if (l < lists && slot < a.k) {
            const int i = l / a.parts, row = row0 + i;
            const int64_t at = ((int64_t)row0 * a.parts + l) * a.k + slot;
            if (a.done && a.done[row]) {
                if (l == i * a.parts && slot == 0) e = Entry{base[i], (uint32_t)i * (uint32_t)a.vocab + (uint32_t)a.end_token};
            } else {
                const float v = a.part_value[at];
                if (v > -__builtin_inff()) e = Entry{base[i] + (double)v, (uint32_t)i * (uint32_t)a.vocab + (uint32_t)a.part_token[at]};
            }
            if (!(e.total > -kInf)) e = Entry{-kInf, ~0u};  // NaN too
        }
        best = merge(best, e, kp, lane);
    }
    best = merge_wave(best, kp, lane);
    if (waves > 1) {
        if (lane < kp) {
            sm_total[wave * kp + lane] = best.total;
            sm_flat[wave * kp + lane] = best.flat;
        }
        __syncthreads();
        if (wave > 0) return;
        best = Entry{-kInf, ~0u};
        for (int w0 = 0; w0 < waves; w0 += per) {
            Entry e{-kInf, ~0u};
            const int w = w0 + lane / kp;
            if (w < waves) e = Entry{sm_total[w * kp + slot], sm_flat[w * kp + slot]};
            best = merge(best, e, kp, lane);
        }
        best = merge_wave(best, kp, lane);
    }
    if (wave == 0 && lane < a.k) {
        const int64_t at = (int64_t)blockIdx.x * a.k + lane;
        const bool real = best.flat != ~0u;
        const uint32_t beam = real ? best.flat / (uint32_t)a.vocab : (uint32_t)min(lane, a.beams - 1);
        a.out_scores[at] = (float)best.total;
        a.out_parents[at] = (int32_t)beam;
        a.out_tokens[at] = real ? (int32_t)(best.flat - beam * (uint32_t)a.vocab) : -1;
    }
}

// Vectors a lane: 16 where that still gives the chip its waves, else 4, so that a few rows spread over it
int vectors(int64_t rows, int64_t vocab, fp4_dtype xt)
{
    const int64_t part = 64 * 16 * (xt == FP4_BF16 ? 8 : 4);
    return rows * ((vocab + part - 1) / part) >= 2048 ? 16 : 4;
}

}  // namespace

int64_t beam_parts(int64_t rows, int64_t vocab, fp4_dtype xt)
{
    const int64_t part = 64 * (xt == FP4_BF16 ? 8 : 4) * vectors(rows, vocab, xt);
    return (vocab + part - 1) / part;
}

fp4_status launch_beam_select(BeamArgs a, fp4_dtype xt, hipStream_t st)
{
    const int64_t rows = (int64_t)a.batch * a.beams;
    a.parts = (int)beam_parts(rows, a.vocab, xt);
    const int nv = vectors(rows, a.vocab, xt);
    const dim3 grid((unsigned)((rows * a.parts + 3) / 4));
    if (xt == FP4_BF16) {
        if (nv == 16) hipLaunchKernelGGL((k_beam_rows<uint16_t, 16>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_beam_rows<uint16_t, 4>), grid, dim3(256), 0, st, a);
    } else {
        if (nv == 16) hipLaunchKernelGGL((k_beam_rows<float, 16>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_beam_rows<float, 4>), grid, dim3(256), 0, st, a);
    }
    int kp = 1;
    while (kp < a.k) kp <<= 1;
    const int64_t steps = ((int64_t)a.beams * a.parts * kp + 63) / 64;  // of one wave
    const int waves = steps >= 32 ? 16 : steps >= 8 ? 4 : 1;
    hipLaunchKernelGGL(k_beam_join, dim3((unsigned)a.batch), dim3(64 * waves), 0, st, a, kp);
    return hipGetLastError() == hipSuccess ? FP4_OK : FP4_ERR_HIP;
}

}  // namespace fp4k
