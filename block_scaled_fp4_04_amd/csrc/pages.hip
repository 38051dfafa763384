// pages.hip -- pages of the key-value cache dealt and taken back on the device: block tables, slots and
// positions from request lengths, the free list from the tables that are alive, block tables and partly
// filled pages of beams after a selection.  (quant.hip fills the slots, the attention kernels read the tables.)
//
// All of it is a few integers a sequence, a token or a table entry: bound by the launch and by chains of
// dependent loads and scans, not by bytes, so the small calls are one workgroup and one launch (64 sequences of one token
// 3.1 us; 300 sequences and 32000 tokens in two launches 4.6 + 3.1 us; the free list of 26000 pages from 512 rows
// 4.4 + 5.0 us; tables of 288 beams 4.9 us and their page copies 5.3 us).  Results do not depend on
// the order of workgroups: sums are prefix sums, and no entry is written by one workgroup and read by another
// of the same launch.
#include "device_common.h"
#include "internal.h"

namespace fp4k {

namespace {

constexpr uint32_t kFull = 0x7FFFFFFFu;  // sums saturate here, so that bad lengths cannot wrap

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b)
{
    const uint32_t s = a + b;  // both at most kFull
    return s > kFull ? kFull : s;
}

// lane i takes lane i - SHIFT's value of its row of 16 (0 where there is none), or the last one of the row or the two
// rows before
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t before(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}

// Inclusive prefix sum over the workgroup's threads (saturating sums of non-negative numbers are
// associative).  `red` holds one value a wave; `total` is the sum of all.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *red, uint32_t &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    v = sat_add(v, before<0x111, 0xF>(v));  // row_shr 1, 2, 4, 8
    v = sat_add(v, before<0x112, 0xF>(v));
    v = sat_add(v, before<0x114, 0xF>(v));
    v = sat_add(v, before<0x118, 0xF>(v));
    v = sat_add(v, before<0x142, 0xA>(v));  // rows 1 and 3 take the last of rows 0 and 2
    v = sat_add(v, before<0x143, 0xC>(v));  // rows 2 and 3 that of row 1
    if (waves == 1) {
        total = (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
        return v;
    }
    __syncthreads();  // the last scan's readers
    if (lane == 63) red[wave] = v;
    __syncthreads();
    uint32_t before = 0, sum = 0;
    for (int w = 0; w < waves; ++w) {
        if (w == wave) before = sum;
        sum = sat_add(sum, red[w]);
    }
    total = sum;
    return sat_add(v, before);
}

// What the tokens of a sequence need to find their slots
struct Span {
    uint32_t end;    // its last new token + 1 in the packed batch
    int32_t held;    // its length before
    int32_t fresh;   // its place in the order of new pages; -1: refused
};

// One workgroup over all sequences (pages that a refused one asked for stay in the running sum, so that nobody overtakes
// it): Span s to `spans`, lengths, offsets and the pool's state written.
// Returns the free pages before the call.
__device__ __forceinline__ int32_t deal_pages(const PageArgs &a, Span *spans)
{
    __shared__ uint32_t red[16];
    __shared__ uint32_t sm_taken, sm_refused;
    if (threadIdx.x == 0) sm_taken = sm_refused = 0;
    const int32_t state0 = a.state_in[0], state1 = a.state_in[1];
    const int32_t count = min(max(state0, 0), a.pages);
    const int64_t room = (int64_t)a.width << a.page_shift;
    uint32_t new0 = 0, page0 = 0, len0 = 0;  // sums over the chunks before
    __syncthreads();
    for (int base = 0; base < a.seqs; base += blockDim.x) {
        const int b = base + (int)threadIdx.x;
        const bool is = b < a.seqs;
        const int32_t held = is ? a.seq_lens[b] : 0;
        const int32_t want = is ? max(a.new_lens[b], 0) : 0;
        uint32_t total;
        const uint32_t end = sat_add(new0, block_scan((uint32_t)want, red, total));
        new0 = sat_add(new0, total);
        const int64_t len = (int64_t)held + want;
        const bool fits = is && held >= 0 && len <= room && end <= (uint32_t)a.tokens;
        const int32_t page = 1 << a.page_shift;
        const int32_t have = fits ? (int32_t)(((int64_t)held + page - 1) >> a.page_shift) : 0;
        const int32_t need = fits ? (int32_t)((len + page - 1) >> a.page_shift) - have : 0;
        const uint32_t upto = sat_add(page0, block_scan((uint32_t)need, red, total));
        page0 = sat_add(page0, total);
        const bool given = fits && (need == 0 || upto <= (uint32_t)count);
        const int32_t now = given ? held + want : held;
        const uint32_t lens = sat_add(len0, block_scan((uint32_t)max(now, 0), red, total));
        len0 = sat_add(len0, total);
        if (given && need > 0) atomicMax(&sm_taken, upto);
        if (is && !given && want > 0) atomicAdd(&sm_refused, 1u);
        if (is) {
            spans[b] = Span{end, held, given ? (int32_t)(upto - need) : -1};
            a.lens_out[b] = now;
            if (a.cu_q) a.cu_q[b + 1] = (int32_t)min(end, (uint32_t)a.tokens);
            if (a.cu_k) a.cu_k[b + 1] = (int32_t)lens;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        a.state_out[0] = count - (int32_t)sm_taken;
        a.state_out[1] = state1 + (int32_t)sm_refused;
        if (a.cu_q) a.cu_q[0] = 0;
        if (a.cu_k) a.cu_k[0] = 0;
    }
    return count;
}

// Slot, position and, where it begins a page, table entry of new token t of sequence b
__device__ __forceinline__ void place_token(const PageArgs &a, const Span *spans, int32_t count, uint32_t t, int b)
{
    int64_t slot = -1;
    int32_t pos = 0;
    if (b < a.seqs) {
        const Span s = spans[b];
        const uint32_t begin = b > 0 ? spans[b - 1].end : 0u;
        pos = (int32_t)((uint32_t)s.held + (t - begin));
        if (s.fresh >= 0) {
            const int32_t at = pos >> a.page_shift;
            const int32_t have = (int32_t)(((int64_t)s.held + (1 << a.page_shift) - 1) >> a.page_shift);
            const int32_t fresh = at - have;
            int32_t *entry = a.table + b * a.table_stride + at;
            int32_t id;
            if (fresh >= 0) {
                id = a.free_list[count - 1 - s.fresh - fresh];
                if ((pos & ((1 << a.page_shift) - 1)) == 0) *entry = id;
            } else {
                id = *entry;
            }
            if (id >= 0 && id < a.pages) slot = ((int64_t)id << a.page_shift) | (pos & ((1 << a.page_shift) - 1));
        }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
}

// the first sequence whose new tokens end past t (in LDS, a search a lane)
__device__ __forceinline__ int span_of(const Span *spans, int seqs, uint32_t t)
{
    int lo = 0, hi = seqs;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (spans[mid].end > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// One workgroup, one launch, up to these sizes (one / two launches, the host's part of a launch, 3 us, aside: 64 sequences of
// 1 token 2.6 / 5.3 us, of 16 6.6 / 6.0, of 64 9.2 / 6.2; one of 2048 5.2 / 4.2, of 8192 8.3 / 4.3; 1000 of 1 5.5 / 8.5)
constexpr int kSmallSeqs = 1024, kSmallTokens = 2048;

// Everything in one workgroup
__global__ __launch_bounds__(1024) void k_pages_extend_small(PageArgs a)
{
    __shared__ Span spans[kSmallSeqs];
    const int32_t count = deal_pages(a, spans);
    __syncthreads();
    for (uint32_t t = threadIdx.x; t < (uint32_t)a.tokens; t += blockDim.x)
        place_token(a, spans, count, t, span_of(spans, a.seqs, t));
}

// Two launches: the sequences in one workgroup, then the tokens
__global__ __launch_bounds__(1024) void k_pages_deal(PageArgs a)
{
    Span *spans = reinterpret_cast<Span *>(a.ws + 4);
    const int32_t count = deal_pages(a, spans);
    if (threadIdx.x == 0) a.ws[0] = count;
}

// The same in memory for the 64 consecutive tokens of a wave: 64 ends at a time down to the first token's, then those behind
// it (300 sequences, 32000 tokens: 4.6 us with a search a lane, 3.3 us; in LDS the search a lane is the faster one, 2.6
// against 4.2 us for 64 tokens)
__device__ __forceinline__ int wave_span_of(const Span *spans, int seqs, uint32_t t)
{
    const int lane = threadIdx.x & 63;
    const uint32_t t0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)t);
    int lo = 0;
    for (int span = seqs; span > 0;) {  // the answer for t0 is in [lo, lo + span]
        const int step = (span + 63) >> 6, at = lo + (lane + 1) * step - 1;
        const bool past = at < lo + span && spans[at].end <= t0;
        const int skip = __builtin_popcountll(__ballot(past)) * step;
        lo += skip;
        span = min(step - 1, span - skip);
    }
    int b = lo;
    for (int base = lo; base < seqs; base += 64) {
        const uint32_t end = base + lane < seqs ? spans[base + lane].end : kFull;
        const uint64_t over = __ballot(end > t0 + 63);  // past the last lane's token
        const int n = over ? __builtin_ctzll(over) : 64;
        for (int i = 0; i < n; ++i) b += (uint32_t)__builtin_amdgcn_readlane((int)end, i) <= t;
        if (over) break;
    }
    return b;
}

__global__ __launch_bounds__(256) void k_pages_place(PageArgs a)
{
    const Span *spans = reinterpret_cast<const Span *>(a.ws + 4);
    const uint32_t t = blockIdx.x * 256u + threadIdx.x;
    const int b = wave_span_of(spans, a.seqs, t);
    if (t < (uint32_t)a.tokens) place_token(a, spans, a.ws[0], t, b);
}

// ------------------------------------------------- pages nobody holds --
//
// A bitmap of the pages that some row holds, in LDS; what is left, in ascending order, is the free
// list.  Bits are set with LDS atomics (or: the order does not matter).

constexpr int kRangeWords = 8192, kRangePages = kRangeWords * 32;  // 32 KiB of LDS

// The rows of wave `wave` of `waves`: as many at a time as fit its lanes (a row takes a power of two of them, up to all),
// four such steps in flight.
__device__ __forceinline__ void mark_pages(const PageArgs &a, uint32_t *bits, int32_t low, int wave, int waves)
{
    constexpr int U = 4;
    const int lane = threadIdx.x & 63;
    int span = 1;
    while (span < a.width && span < 64) span <<= 1;
    const int once = 64 / span, col = lane & (span - 1);
    auto mark = [&](int32_t id) {
        if (id >= 0 && id < a.pages && id >= low && id < low + kRangePages) atomicOr(&bits[(id - low) >> 5], 1u << ((id - low) & 31));
    };
    for (int64_t b0 = (int64_t)wave * once; b0 < a.seqs; b0 += (int64_t)U * waves * once) {
        int entries[U];
        const int32_t *row[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t b = b0 + (int64_t)u * waves * once + lane / span;
            const int64_t n = b < a.seqs ? (int64_t)max(a.seq_lens[b], 0) + (1 << a.page_shift) - 1 : 0;
            entries[u] = (int)min(n >> a.page_shift, (int64_t)a.width);
            row[u] = a.table + b * a.table_stride;
        }
        int32_t id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = col < entries[u] ? row[u][col] : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) mark(id[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
            for (int i = col + 64; i < entries[u]; i += 256) {  // (wider rows take all lanes)
                int32_t more[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) more[c] = i + 64 * c < entries[u] ? row[u][i + 64 * c] : -1;
#pragma unroll
                for (int c = 0; c < 4; ++c) mark(more[c]);
            }
    }
}

// 32 pages a thread, `held` its word (all ones past the pool): free ids from place `at` on.  A wave
// writes two words' ids at a time, as far as a word has any.
__device__ __forceinline__ void list_pages(const PageArgs &a, uint32_t held, int32_t first, uint32_t at)
{
    const int lane = threadIdx.x & 63, half = lane >> 5, bit = lane & 31;
    const uint32_t open = ~held;
    const uint64_t some = __ballot(open != 0);
    const int words = some ? 64 - __builtin_clzll(some) : 0;
    for (int i = 0; i < words; i += 8) {
        uint32_t w[4], p[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            w[u] = __shfl(open, i + 2 * u + half, kWave);
            p[u] = __shfl(at, i + 2 * u + half, kWave);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if ((w[u] >> bit) & 1u) a.free_list[p[u] + __builtin_popcount(w[u] & ((1u << bit) - 1u))] = first + (i + 2 * u) * 32 + lane;
    }
}

// bits past the pool count as held
__device__ __forceinline__ uint32_t pool_word(uint32_t w, int64_t first, int64_t pages)
{
    if (first >= pages) return ~0u;
    return pages - first < 32 ? w | (~0u << (int)(pages - first)) : w;
}

__global__ __launch_bounds__(1024) void k_pages_collect_small(PageArgs a)
{
    __shared__ uint32_t bits[kRangeWords];
    __shared__ uint32_t red[16];
    const int words = (a.pages + 31) >> 5;
    for (int i = threadIdx.x; i < words; i += blockDim.x) bits[i] = 0;
    __syncthreads();
    mark_pages(a, bits, 0, threadIdx.x >> 6, blockDim.x >> 6);
    __syncthreads();
    uint32_t done = 0, total;
    for (int base = 0; base < words; base += blockDim.x) {
        const int i = base + (int)threadIdx.x;
        const uint32_t w = pool_word(i < words ? bits[i] : ~0u, (int64_t)i * 32, a.pages);
        const uint32_t n = __builtin_popcount(~w);
        const uint32_t upto = block_scan(n, red, total);
        list_pages(a, w, (i & ~63) * 32, done + upto - n);
        done += total;
    }
    if (threadIdx.x == 0) a.state_out[0] = (int32_t)done;
}

// Large pools and tables: grid (parts, ranges); a part of the rows marks one range of the pages.  The bitmap of
// part p is at ws + p * words.
constexpr int kMarkParts = 16;

__global__ __launch_bounds__(1024) void k_pages_mark(PageArgs a, int64_t words)
{
    __shared__ uint32_t bits[kRangeWords];
    const int64_t word0 = (int64_t)blockIdx.y * kRangeWords;
    const int n = (int)min(words - word0, (int64_t)kRangeWords), waves = blockDim.x >> 6;
    for (int i = threadIdx.x; i < n; i += blockDim.x) bits[i] = 0;
    __syncthreads();
    mark_pages(a, bits, (int32_t)(word0 * 32), (int)blockIdx.x * waves + (int)(threadIdx.x >> 6), (int)gridDim.x * waves);
    __syncthreads();
    uint32_t *out = reinterpret_cast<uint32_t *>(a.ws) + blockIdx.x * words + word0;
    for (int i = threadIdx.x; i < n; i += blockDim.x) out[i] = bits[i];
}

__device__ __forceinline__ uint32_t marked(const uint32_t *ws, int64_t words, int64_t i)
{
    uint32_t w = 0;
#pragma unroll
    for (int p = 0; p < kMarkParts; ++p) w |= ws[p * words + i];
    return w;
}

// One workgroup a 1024 words: what is free before them, then their own.  (Quadratic in the pool: of 4194304 pages the whole call
// takes 102 us, of 16777216 827.)
__global__ __launch_bounds__(1024) void k_pages_sweep(PageArgs a, int64_t words)
{
    __shared__ uint32_t red[16];
    const uint32_t *ws = reinterpret_cast<const uint32_t *>(a.ws);
    const int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x;
    const uint32_t w = i < words ? pool_word(marked(ws, words, i), i * 32, a.pages) : ~0u;
    uint32_t before = 0, base = 0, total;
    for (int64_t j = threadIdx.x; j < (int64_t)blockIdx.x * 1024; j += 1024) before += __builtin_popcount(~marked(ws, words, j));
    if (blockIdx.x > 0) block_scan(before, red, base);
    const uint32_t n = __builtin_popcount(~w), upto = block_scan(n, red, total);
    list_pages(a, w, (int32_t)((i & ~int64_t(63)) * 32), base + upto - n);
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) a.state_out[0] = (int32_t)(base + total);
}

// ------------------------------------------------------------- beams --
//
// Row j of a group takes the row of its parent.  Full pages are shared by the rows that hold them; a
// partly filled page belongs to one row alone, so of several children of a parent the first keeps its
// page and each further one needs a copy.  There are as many further children as rows without a child,
// and the m-th further child takes the page of the m-th such row to copy into: no page is dealt.
// Rows of a group differ in length where a pool ran out under some of them.  Only a row's
// own partly filled page is ever copied into (what its length does not cover may be another sequence's, full
// pages may be shared), and entries that the parent does not give become -1.

constexpr int kTile = 256;  // table columns of a workgroup

// the set bit of `dropped` that has `rank` set bits below it
__device__ __forceinline__ int nth_bit(uint64_t dropped, int rank)
{
    for (; rank > 0; --rank) dropped &= dropped - 1;
    return __builtin_ctzll(dropped);
}

__global__ __launch_bounds__(256) void k_pages_reorder(BeamTableArgs a)
{
    extern __shared__ int32_t tile[];  // [beams][kTile]: read whole before any row is written, so in place is fine
    const int group = (int)blockIdx.x / a.tiles, part = (int)blockIdx.x - group * a.tiles;
    const int64_t row0 = (int64_t)group * a.beams;
    const int col = part * kTile + (int)threadIdx.x, lane = threadIdx.x & 63;
    for (int j = 0; j < a.beams; ++j)
        tile[j * kTile + threadIdx.x] = col < a.width ? a.table[(row0 + j) * a.table_stride + col] : -1;

    // every wave: its lane's row, the rows with a child, the further children
    int parent = lane, own = 0;
    if (lane < a.beams) {
        const int p = a.parents[row0 + lane];
        if (p >= 0 && p < a.beams) parent = p;
        own = max(a.seq_lens[row0 + lane], 0);
    }
    const int len = __shfl(own, parent, kWave);
    uint64_t children = 0;
    bool further = false;
    for (int s = 0; s < a.beams; ++s) {
        const int p = __builtin_amdgcn_readlane(parent, s);
        children |= 1ull << p;
        further |= s < lane && p == parent;
    }
    const uint64_t more = __ballot(further && lane < a.beams);
    const uint64_t dropped = ~children & (~0ull >> (64 - a.beams));  // as many as `more`
    // a further child's row to take the page of (-1: that row has no partly filled page there)
    const int at = len >> a.page_shift, off = len & ((1 << a.page_shift) - 1);
    int spare = further ? nth_bit(dropped, __builtin_popcountll(more & ((1ull << lane) - 1))) : lane;
    if ((uint32_t)(__shfl(own, spare, kWave) - (len - off)) - 1u >= (1u << a.page_shift) - 1u) spare = -1;
    __syncthreads();

    if (threadIdx.x < 64 && lane < a.beams) {
        const bool copied = further && off > 0 && at < a.width && spare >= 0;
        if ((copied ? at / kTile : 0) == part) {  // the workgroup of the last page's column
            int32_t *rec = a.copies + (row0 + lane) * 3;
            int32_t src = -1, dst = -1;
            if (copied) {
                src = tile[parent * kTile + at % kTile];
                dst = tile[spare * kTile + at % kTile];
            }
            rec[0] = src;
            rec[1] = dst;
            rec[2] = copied ? off : 0;
        }
    }
    for (int j = 0; j < a.beams; ++j) {
        const int p = __builtin_amdgcn_readlane(parent, j), n = __builtin_amdgcn_readlane(len, j);
        const int last = n >> a.page_shift, part_of = n & ((1 << a.page_shift) - 1), mine = __builtin_amdgcn_readlane(own, j);
        const bool given = col < last + (part_of > 0);
        if (col >= a.width || !(given || (int64_t)col << a.page_shift < mine)) continue;
        const bool heir = col == last && ((more >> j) & 1ull);
        const int from = !given ? -1 : heir ? __builtin_amdgcn_readlane(spare, j) : p;
        a.out[(row0 + j) * a.out_stride + col] = from >= 0 ? tile[from * kTile + threadIdx.x] : -1;
    }
}

// The first tokens of page copies[i][0] into page copies[i][1]: a workgroup a copy, head and side.
// Codes of consecutive tokens are consecutive bytes; scale bytes are one run of tokens a block.
__global__ __launch_bounds__(256) void k_kv_copy(KvArgs a, const int32_t *copies, int row_bytes, int blocks)
{
    const uint32_t per = 2u * a.kv_heads, i = blockIdx.x / per, hp = blockIdx.x - i * per;
    const int side = hp >= (uint32_t)a.kv_heads, head = (int)hp - (side ? a.kv_heads : 0);
    const int32_t src = copies[3 * i], dst = copies[3 * i + 1], page = 1 << a.page_shift;
    const int32_t tokens = min(copies[3 * i + 2], page);
    if (src < 0 || dst < 0 || src >= a.pages || dst >= a.pages || src == dst || tokens <= 0) return;
    const int64_t from = ((int64_t)src * a.kv_heads + head) << a.page_shift, to = ((int64_t)dst * a.kv_heads + head) << a.page_shift;
    uint8_t *codes = side ? a.codes[1] : a.codes[0], *scales = side ? a.scales[1] : a.scales[0];
    const uint4 *x = reinterpret_cast<const uint4 *>(codes + from * row_bytes);
    uint4 *y = reinterpret_cast<uint4 *>(codes + to * row_bytes);
    const int n = (tokens * row_bytes) >> 4;  // rows are multiples of 32 bytes
    for (int j = threadIdx.x; j < n; j += 256) y[j] = x[j];
    if (blocks == 0) return;
    const uint8_t *u = scales + from * blocks;
    uint8_t *w = scales + to * blocks;
    const int words = page >> 4;  // 16 tokens' bytes
    for (int j = threadIdx.x; j < blocks * words; j += 256) {
        const int t0 = (j & (words - 1)) << 4;
        if (t0 + 16 <= tokens) reinterpret_cast<uint4 *>(w)[j] = reinterpret_cast<const uint4 *>(u)[j];
        else
            for (int t = t0; t < tokens; ++t) w[j * 16 + t - t0] = u[j * 16 + t - t0];
    }
}

unsigned whole_waves(int64_t n) { return n >= 1024 ? 1024u : n <= 64 ? 64u : (unsigned)((n + 63) & ~int64_t(63)); }

}  // namespace

bool pages_extend_small(int64_t seqs, int64_t tokens) { return seqs <= kSmallSeqs && tokens <= kSmallTokens; }

size_t pages_extend_bytes(int64_t seqs, int64_t tokens)
{
    return pages_extend_small(seqs, tokens) ? 0 : align256(16 + (size_t)seqs * sizeof(Span));
}

fp4_status launch_pages_extend(const PageArgs &a, hipStream_t st)
{
    if (pages_extend_small(a.seqs, a.tokens)) {
        const int64_t n = a.seqs > a.tokens ? a.seqs : a.tokens;
        hipLaunchKernelGGL(k_pages_extend_small, dim3(1), dim3(whole_waves(n)), 0, st, a);
    } else {
        hipLaunchKernelGGL(k_pages_deal, dim3(1), dim3(whole_waves(a.seqs)), 0, st, a);
        if (a.tokens > 0) hipLaunchKernelGGL(k_pages_place, dim3((unsigned)((a.tokens + 255) / 256)), dim3(256), 0, st, a);
    }
    return hipGetLastError() == hipSuccess ? FP4_OK : FP4_ERR_HIP;
}

// One workgroup, one launch, for small tables and pools that fit its bitmap (one / two launches, the host's part of a launch aside:
// tables of 16 x 16 entries 3.4 / 4.3 us, 64 x 64 5.6 / 6.7, 64 x 128 7.1 / 7.2, 256 x 64 9.1 / 7.0, 512 x 512 52 / 14)
static bool collect_small(int64_t pages, int64_t seqs, int64_t width) { return pages <= kRangePages && seqs * width <= 8192; }

size_t pages_collect_bytes(int64_t pages, int64_t seqs, int64_t width)
{
    return collect_small(pages, seqs, width) ? 0 : align256((size_t)kMarkParts * ((pages + 31) / 32) * 4);
}

fp4_status launch_pages_collect(const PageArgs &a, hipStream_t st)
{
    if (collect_small(a.pages, a.seqs, a.width)) {
        hipLaunchKernelGGL(k_pages_collect_small, dim3(1), dim3(1024), 0, st, a);
    } else {
        const int64_t words = ((int64_t)a.pages + 31) / 32;
        hipLaunchKernelGGL(k_pages_mark, dim3(kMarkParts, (unsigned)((words + kRangeWords - 1) / kRangeWords)), dim3(1024), 0, st, a, words);
        hipLaunchKernelGGL(k_pages_sweep, dim3((unsigned)((words + 1023) / 1024)), dim3(1024), 0, st, a, words);
    }
    return hipGetLastError() == hipSuccess ? FP4_OK : FP4_ERR_HIP;
}

int64_t pages_reorder_grid(int64_t batch, int64_t width) { return batch * ((width + kTile - 1) / kTile); }

fp4_status launch_pages_reorder(BeamTableArgs a, hipStream_t st)
{
    a.tiles = (a.width + kTile - 1) / kTile;
    hipLaunchKernelGGL(k_pages_reorder, dim3((unsigned)pages_reorder_grid(a.batch, a.width)), dim3(kTile),
                       (size_t)a.beams * kTile * 4, st, a);
    return hipGetLastError() == hipSuccess ? FP4_OK : FP4_ERR_HIP;
}

fp4_status launch_kv_copy(const KvArgs &a, fp4_kv_format fmt, const int32_t *copies, int64_t n, hipStream_t st)
{
    const int row = fmt == FP4_KV_BF16 ? 2 * a.head_dim : fmt == FP4_KV_MXFP8 ? a.head_dim : a.head_dim / 2;
    const int blocks = fmt == FP4_KV_BF16 ? 0 : a.head_dim / (fmt == FP4_KV_NVFP4 ? 16 : 32);
    hipLaunchKernelGGL(k_kv_copy, dim3((unsigned)(n * 2 * a.kv_heads)), dim3(256), 0, st, a, copies, row, blocks);
    return hipGetLastError() == hipSuccess ? FP4_OK : FP4_ERR_HIP;
}

}  // namespace fp4k
