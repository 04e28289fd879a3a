// Rows of a table looked up by token, and the table's gradient.
//
//   out[i] = scale * table[k_i]
//   dw[v] (+)= scale * sum of dy[i] over the i with k_i = v, in ascending order
//
// Both move memory and compute next to nothing.  The gradient goes by tokens
// sorted by vocabulary row, so that every row is summed in float32 in one
// place and written once; no float atomics, so results are the same each time.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "df11.h"
#include "df11_elements.h"
#include "df11_launch.h"

#pragma clang fp contract(off)

namespace {

using namespace df11_detail;

struct LookupArgs {
    const void *table, *tokens;
    void *out;
    uint64_t table_stride, out_stride;
    uint32_t n, rows, cols, parts;  // parts: waves of a token
    float scale;
};

// The token's row of the table, or 2^32 - 1 where it has none.
template <class I>
__device__ __forceinline__ uint32_t row_of(I token, uint32_t rows) {
    return token >= 0 && uint64_t(token) < rows ? uint32_t(token) : 0xFFFFFFFFu;
}

// ---------------------------------------------------------------- lookup

// The group times `scale`, each product rounded to float32: without the empty
// statement those of two float16 become mixed operations that round only once,
// to the result's type.
__device__ __forceinline__ f32x8 scaled(f32x8 x, float scale) {
    x *= scale;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        float p = x[e];
        asm("" : "+v"(p));
        x[e] = p;
    }
    return x;
}

constexpr uint32_t kAhead = 4;               // groups that a lane has on their way
constexpr uint32_t kPart = 64 * 8 * kAhead;  // columns of a wave

template <class T, class Y, class I>
__global__ __launch_bounds__(256) void lookup(LookupArgs a) {
    const uint32_t wave = uniform(blockIdx.x * 4 + (threadIdx.x >> 6)), lane = threadIdx.x & 63u;
    const uint32_t i = wave / a.parts, c0 = wave % a.parts * kPart + lane * 8;
    if (i >= a.n) return;
    const uint32_t row = row_of(static_cast<const I *>(a.tokens)[i], a.rows);
    Y *out = static_cast<Y *>(a.out) + i * a.out_stride;
    if (row == 0xFFFFFFFFu) {
        const f32x8 nan = f32x8(__builtin_nanf(""));
#pragma unroll
        for (uint32_t u = 0; u < kAhead; u++) store_group<Y>(out, c0 + u * 512, a.cols, nan);
        return;
    }
    const T *from = static_cast<const T *>(a.table) + row * a.table_stride;
    typename Group<T>::type v[kAhead];
#pragma unroll
    for (uint32_t u = 0; u < kAhead; u++) v[u] = load_group<T>(from, c0 + u * 512, a.cols);
#pragma unroll
    for (uint32_t u = 0; u < kAhead; u++) store_group<Y>(out, c0 + u * 512, a.cols, scaled(widen<T>(v[u]), a.scale));
}

// ---------------------------------------------------------------- gradient

// What the launches hand on: the kept tokens sorted by row (each one's position,
// row, and where the run of its row begins and ends), the ends by row of the
// table (0 where there is no token), and sums of runs in chunks.
struct GradArgs {
    const void *tokens, *dy;
    void *dw;
    uint32_t *kept, *total;
    uint4 *sorted;
    float *part;
    uint64_t dy_stride, dw_stride, part_stride;
    int64_t padding;
    uint32_t n, rows, cols, span, run, parts, chunk;
    uint32_t summing;  // workgroups that sum; those behind them clear rows
    float scale;
};

// Calls f(r, which lanes have it, the first of them) for every r of the lanes that
// are `in`.  For counting, LDS atomics are the faster way as long as few lanes can
// have the same r (32768 tokens: 35 against 41 us for the sort), but those on one
// address take their turns (32768 equal tokens: 48 against 31 us).
template <class F>
__device__ __forceinline__ void match(uint32_t r, bool in, F f) {
    for (uint64_t left = __ballot(in); left;) {
        const uint32_t first = __builtin_ctzll(left);
        const uint32_t r0 = __builtin_amdgcn_readlane(r, first);
        const uint64_t same = __ballot(in && r == r0);
        f(r0, same, first);
        left &= ~same;
    }
}

constexpr uint32_t kSortWaves = 16;

// Sorts the tokens by row, stably, in one launch without a word between its
// workgroups: each owns `run` neighbouring rows, reads all tokens twice, and
// keeps those of its rows.  The first reading counts them by wave and row, and
// all tokens of earlier rows, which says where its rows begin; the second puts
// each at its place.  A wave reads `span` consecutive tokens, in order, so
// places within a row ascend with the position.  12 us for 8192 and 31 to 36 us
// for 32768 tokens of 128256 rows.
template <class I>
__global__ __launch_bounds__(64 * kSortWaves) void sort_tokens(GradArgs a) {
    extern __shared__ uint32_t shared[];
    uint32_t *count = shared, *before = shared + kSortWaves * a.run;  // [wave][row], [row]
    __shared__ uint32_t sums[kSortWaves];
    const uint32_t lane = threadIdx.x & 63u, wave = uniform(threadIdx.x >> 6);
    const uint32_t base = blockIdx.x * a.run;
    for (uint32_t i = threadIdx.x; i < kSortWaves * a.run; i += 64 * kSortWaves) count[i] = 0;
    __syncthreads();

    const uint32_t from = min(a.n, wave * a.span), to = min(a.n, from + a.span);
    const I *tokens = static_cast<const I *>(a.tokens);
    // Calls f(position, row less base, whether the row is the workgroup's, whether it
    // is an earlier one) for a wave's tokens, 64 at a time, in order.  The next
    // tokens are on their way meanwhile.  All workgroups visit all tokens, so a visit's
    // instructions count (32768 tokens of which none is kept: 18 us), and the waves
    // wait for LDS at each token that is.
    constexpr uint32_t kLoads = 8;
    const uint32_t mine_rows = min(a.run, a.rows - base);
    const bool padded = uint64_t(a.padding) <= 0xFFFFFFFFu;
    const auto each = [&](auto f) {
        I now[kLoads], next[kLoads];
        const auto fetch = [&](uint32_t p, I (&t)[kLoads]) {
#pragma unroll
            for (uint32_t u = 0; u < kLoads; u++) t[u] = tokens[min(p + 64 * u + lane, a.n - 1)];
        };
        if (from < to) fetch(from, now);
#pragma unroll 1
        for (uint32_t p = from; p < to; p += 64 * kLoads) {
            if (p + 64 * kLoads < to) fetch(p + 64 * kLoads, next);
#pragma unroll
            for (uint32_t u = 0; u < kLoads; u++) {
                const uint32_t i = p + 64 * u + lane, low = uint32_t(now[u]);
                bool valid = p + 64 * kLoads <= to || i < to;
                if constexpr (sizeof(I) == 8) valid = valid && uint64_t(now[u]) >> 32 == 0;
                if (padded) valid = valid && low != uint32_t(a.padding);
                f(i, low - base, valid && low - base < mine_rows, valid && low < base);
                now[u] = next[u];
            }
        }
    };
    // A wave's counts and places are its own: its LDS operations take effect in order.
    volatile uint32_t *place = count + wave * a.run;
    uint32_t below = 0;
    each([&](uint32_t, uint32_t r, bool in, bool earlier) {
        below += __popcll(__ballot(earlier));
        if (__popcll(__ballot(in)) <= 8) {
            if (in) atomicAdd(&count[wave * a.run + r], 1u);
        } else {
            match(r, in, [&](uint32_t r0, uint64_t same, uint32_t first) {
                if (lane == first) place[r0] = place[r0] + __popcll(same);
            });
        }
    });
    if (lane == 0) sums[wave] = below;
    __syncthreads();
    uint32_t start = 0;  // of the workgroup's rows
#pragma unroll
    for (uint32_t w = 0; w < kSortWaves; w++) start += sums[w];
    __syncthreads();

    // counts to places: rows in order (a thread each), the waves of a row in order
    uint32_t mine = 0;
    if (threadIdx.x < a.run)
        for (uint32_t w = 0; w < kSortWaves; w++) mine += count[w * a.run + threadIdx.x];
    uint32_t upto = mine;
#pragma unroll
    for (uint32_t d = 1; d < 64; d <<= 1) {
        const uint32_t other = __shfl_up(upto, d);
        if (lane >= d) upto += other;
    }
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    for (uint32_t w = 0; w < wave; w++) upto += sums[w];
    upto += start;
    if (threadIdx.x < a.run) {
        before[threadIdx.x] = upto;
        if (base + threadIdx.x < a.rows) a.total[base + threadIdx.x] = mine ? upto : 0;
        uint32_t at = upto - mine;
        for (uint32_t w = 0; w < kSortWaves; w++) {
            const uint32_t c = count[w * a.run + threadIdx.x];
            count[w * a.run + threadIdx.x] = at;
            at += c;
        }
        if (blockIdx.x == gridDim.x - 1 && threadIdx.x == a.run - 1) *a.kept = upto;
    }
    __syncthreads();

    each([&](uint32_t i, uint32_t r, bool in, bool) {
        match(r, in, [&](uint32_t r0, uint64_t same, uint32_t first) {
            const uint32_t at = place[r0];
            if (in && r == r0)
                a.sorted[at + __popcll(same & ((1ull << lane) - 1))] =
                    make_uint4(i, base + r, r0 ? before[r0 - 1] : start, before[r0]);
            if (lane == first) place[r0] = at + __popcll(same);
        });
    });
}

template <class Y>
__device__ __forceinline__ Y *row_of_dw(const GradArgs &a, uint32_t row) {
    return static_cast<Y *>(a.dw) + row * a.dw_stride;
}

// Stores a row's sum, added to `old` where ADD.
template <class Y, bool ADD, bool PAST = false>
__device__ __forceinline__ void finish(const GradArgs &a, uint32_t row, uint32_t c, f32x8 sum,
                                       typename Group<Y>::type old) {
    sum = scaled(sum, a.scale);
    if (ADD) sum += widen<Y>(old);
    store_group<Y, PAST>(row_of_dw<Y>(a, row), c, a.cols, sum);
}

template <class Y, bool ADD>
__device__ __forceinline__ void finish(const GradArgs &a, uint32_t row, uint32_t c, f32x8 sum) {
    typename Group<Y>::type old{};
    if (ADD) old = load_group<Y>(row_of_dw<Y>(a, row), c, a.cols);
    finish<Y, ADD>(a, row, c, sum, old);
}

// Clears a wave's 512 columns of a row, `first` and on.
template <class Y, bool PAST>
__device__ __forceinline__ void clear_row(Y *dw, uint32_t first, uint32_t lane, uint32_t cols) {
    if constexpr (sizeof(Y) == 2) {
        store_group<Y, PAST>(dw, first + lane * 8, cols, f32x8(0.0f));
    } else {
        // two halves, each in whole lines, so that these can pass the caches
        typedef f32x4 any __attribute__((aligned(4)));
#pragma unroll
        for (uint32_t half = 0; half < 2; half++) {
            const uint32_t c = first + half * 256 + lane * 4;
            if (c + 4 <= cols) {
                if (PAST) __builtin_nontemporal_store(any(0.0f), reinterpret_cast<any *>(dw + c));
                else *reinterpret_cast<any *>(dw + c) = any(0.0f);
            } else {
#pragma unroll
                for (uint32_t e = 0; e < 3; e++)
                    if (c + e < cols) dw[c + e] = Y(0.0f);
            }
        }
    }
}

// Clears the rows without a token among 64 rows, 512 columns of them.
template <class Y, bool PAST>
__device__ __forceinline__ void clear_rows(const GradArgs &a, uint32_t wave, uint32_t lane) {
    const uint32_t first = wave / a.parts * 64, row = first + lane;
    for (uint64_t none = __ballot(row < a.rows && a.total[min(row, a.rows - 1)] == 0); none; none &= none - 1)
        clear_row<Y, PAST>(row_of_dw<Y>(a, first + __builtin_ctzll(none)), wave % a.parts * 512, lane, a.cols);
}

// Sums the runs of equal rows, a wave for 512 columns of a chunk of sorted tokens:
// the runs that begin in it, also where they go on behind it.  A run longer than
// a chunk is summed by all chunks that it touches; each leaves its sum in the
// chunk's first (the run began before) or second slot.  Without ADD further
// workgroups clear the rows without a token meanwhile.  Bound by HBM.
//
// BIG: what would fill the caches passes them by.  With ADD that is a dy which the
// last cache cannot hold (32768 tokens, added to 128256 rows of float32, the same each
// time, so that dw may stay there: 8192 columns 273 -> 256 us for the three launches,
// 4096 columns 194 -> 172; other inputs each time: 268 and 197 either way).  One that
// it holds is read there if it was made before (66000 tokens, 4001 x 1024: 157 us, past
// the caches 201).  Without ADD it is dw, which leaves dy there (8192 tokens, 128256 x
// 4096 in BF16: 241 -> 212 us; with dy read past the caches as well 240), if of 2 bytes
// an element: a lane stores 8 float32 in two halves, which the caches have to bring
// together (the same in float32: 448 us, past the caches 1000); cleared rows are stored
// otherwise (402 us).
template <class X, class Y, bool ADD, bool BIG>
__global__ __launch_bounds__(256) void sum_runs(GradArgs a) {
    constexpr bool PAST = BIG && !ADD && sizeof(Y) == 2, ONCE = BIG && ADD;
    const uint32_t lane = threadIdx.x & 63u;
    if (!ADD && blockIdx.x >= a.summing)
        return clear_rows<Y, BIG>(a, uniform((blockIdx.x - a.summing) * 4 + (threadIdx.x >> 6)), lane);
    const uint32_t wave = uniform(blockIdx.x * 4 + (threadIdx.x >> 6));
    const uint32_t chunk = wave / a.parts, c = wave % a.parts * 512 + lane * 8;
    const uint32_t kept = *a.kept, begin = chunk * a.chunk;
    if (begin >= kept) return;
    const uint32_t end = min(kept, begin + a.chunk);
    const uint4 first = a.sorted[begin], last = a.sorted[end - 1];
    const uint32_t from = first.z < begin && first.w - first.z <= a.chunk ? first.w : begin;
    const uint32_t to = last.z >= begin && last.w - last.z <= a.chunk ? last.w : end;
    const X *dy = static_cast<const X *>(a.dy);
    constexpr uint32_t kLoads = 8;
    f32x8 sum = 0.0f;
    for (uint32_t j = from; j < to; j += kLoads) {
        typename Group<X>::type v[kLoads];
        typename Group<Y>::type old[kLoads];
        uint4 of[kLoads];
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++) {
            of[u] = a.sorted[min(j + u, to - 1)];
            v[u] = load_group<X, ONCE>(dy + of[u].x * a.dy_stride, c, a.cols);
            // what the sums are added to comes with them
            if (ADD && j + u + 1 == of[u].w) old[u] = load_group<Y>(row_of_dw<Y>(a, of[u].y), c, a.cols);
        }
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++) {
            if (j + u >= to) break;
            sum += widen<X>(v[u]);
            if (j + u + 1 < to && j + u + 1 != of[u].w) continue;
            // the run's last token here
            if (of[u].w - of[u].z > a.chunk) {
                float *part = a.part + (2 * uint64_t(chunk) + (of[u].z < begin ? 0 : 1)) * a.part_stride + c;
                if (c < a.cols) *reinterpret_cast<f32x8 *>(part) = sum;
            } else {
                finish<Y, ADD, PAST>(a, of[u].y, c, sum, old[u]);
            }
            sum = 0.0f;
        }
    }
}

// Joins the sums of a run longer than a chunk, where it begins: a workgroup for 512
// columns, each of its waves a part of the chunks.
template <class Y, bool ADD>
__global__ __launch_bounds__(256) void join_runs(GradArgs a) {
    __shared__ float part_s[3][512];
    const uint32_t wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63u;
    const uint32_t chunk = blockIdx.x / a.parts, c = blockIdx.x % a.parts * 512 + lane * 8;
    const uint32_t kept = *a.kept, begin = chunk * a.chunk;
    if (begin >= kept) return;
    const uint4 of = a.sorted[min(kept, begin + a.chunk) - 1];
    if (of.z < begin || of.w - of.z <= a.chunk) return;
    // the run's chunks behind this one; slot 1 of this one and slot 0 of those
    const uint32_t chunks = (of.w - 1) / a.chunk - chunk, from = chunks * wave / 4, to = chunks * (wave + 1) / 4;
    const float *part = a.part + 2 * uint64_t(chunk + 1) * a.part_stride + min(c, uint32_t(a.part_stride) - 8);
    constexpr uint32_t kLoads = 8;
    f32x8 sum = 0.0f;
    if (wave == 0) sum = *reinterpret_cast<const f32x8 *>(part - a.part_stride);
    for (uint32_t k = from; k < to; k += kLoads) {
        f32x8 v[kLoads];
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++)
            v[u] = *reinterpret_cast<const f32x8 *>(part + 2 * uint64_t(min(k + u, to - 1)) * a.part_stride);
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++)
            if (k + u < to) sum += v[u];
    }
    if (wave) *reinterpret_cast<f32x8 *>(&part_s[wave - 1][lane * 8]) = sum;
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (uint32_t w = 0; w < 3; w++) sum += *reinterpret_cast<const f32x8 *>(&part_s[w][lane * 8]);
    finish<Y, ADD>(a, of.y, c, sum);
}

// Few tokens: all of it in one launch.  A workgroup owns `run` neighbouring rows
// and 512 columns of them, sorts its rows' tokens in LDS and sums them; a row of
// many tokens is shared by its waves.  2048 tokens are 4 for each of its threads,
// which hold them in registers.  300 tokens, 1999 x 513: 10 us on the GPU where the
// three launches above take 18.
constexpr uint32_t kFew = 2048, kFewWaves = 8, kFewEach = kFew / (64 * kFewWaves), kFewRows = 256;
constexpr uint32_t kMany = 16;  // tokens of a row that its waves share

// The sum of dy over the listed positions, columns c .. c + 7.
template <class X>
__device__ __forceinline__ f32x8 sum_listed(const GradArgs &a, const uint16_t *list, uint32_t n, uint32_t c) {
    const X *dy = static_cast<const X *>(a.dy);
    constexpr uint32_t kLoads = 8;
    f32x8 sum = 0.0f;
    for (uint32_t j = 0; j < n; j += kLoads) {
        typename Group<X>::type v[kLoads];
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++)
            v[u] = load_group<X>(dy + uniform(list[min(j + u, n - 1)]) * a.dy_stride, c, a.cols);
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++)
            if (j + u < n) sum += widen<X>(v[u]);
    }
    return sum;
}

template <class X, class Y, class I, bool ADD>
__global__ __launch_bounds__(64 * kFewWaves) void sum_few(GradArgs a) {
    __shared__ uint32_t count[kFewWaves][kFewRows], end[kFewRows];
    __shared__ uint16_t list[kFew];
    __shared__ uint32_t sums[kFewWaves];
    __shared__ float part[kFewWaves][512];
    const uint32_t lane = threadIdx.x & 63u, wave = uniform(threadIdx.x >> 6);
    const uint32_t base = blockIdx.x / a.parts * a.run, c = blockIdx.x % a.parts * 512 + lane * 8;
    for (uint32_t i = threadIdx.x; i < kFewWaves * a.run; i += 64 * kFewWaves) count[i / a.run][i % a.run] = 0;
    // a wave's tokens are consecutive
    uint32_t row[kFewEach];
#pragma unroll
    for (uint32_t u = 0; u < kFewEach; u++) {
        const uint32_t i = wave * a.span + 64 * u + lane;
        const I t = 64 * u < a.span && i < a.n ? static_cast<const I *>(a.tokens)[i] : I(-1);
        row[u] = int64_t(t) == a.padding ? 0xFFFFFFFFu : row_of(t, a.rows);
        row[u] = row[u] - base < a.run && row[u] >= base ? row[u] - base : 0xFFFFFFFFu;
    }
    __syncthreads();
    volatile uint32_t *place = count[wave];
#pragma unroll
    for (uint32_t u = 0; u < kFewEach; u++)
        match(row[u], row[u] != 0xFFFFFFFFu, [&](uint32_t r0, uint64_t same, uint32_t first) {
            if (lane == first) place[r0] = place[r0] + __popcll(same);
        });
    __syncthreads();
    uint32_t mine = 0;
    if (threadIdx.x < a.run)
        for (uint32_t w = 0; w < kFewWaves; w++) mine += count[w][threadIdx.x];
    uint32_t upto = mine;
#pragma unroll
    for (uint32_t d = 1; d < 64; d <<= 1) {
        const uint32_t other = __shfl_up(upto, d);
        if (lane >= d) upto += other;
    }
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    for (uint32_t w = 0; w < wave; w++) upto += sums[w];
    if (threadIdx.x < a.run) {
        end[threadIdx.x] = upto;
        uint32_t at = upto - mine;
        for (uint32_t w = 0; w < kFewWaves; w++) {
            const uint32_t k = count[w][threadIdx.x];
            count[w][threadIdx.x] = at;
            at += k;
        }
    }
    __syncthreads();
#pragma unroll
    for (uint32_t u = 0; u < kFewEach; u++)
        match(row[u], row[u] != 0xFFFFFFFFu, [&](uint32_t r0, uint64_t same, uint32_t first) {
            const uint32_t at = place[r0];
            if (row[u] == r0)
                list[at + __popcll(same & ((1ull << lane) - 1))] = uint16_t(wave * a.span + 64 * u + lane);
            if (lane == first) place[r0] = at + __popcll(same);
        });
    __syncthreads();

    uint64_t many = 0;  // whether a row of many tokens is among the workgroup's
    for (uint32_t r = wave; r < a.run && base + r < a.rows; r += kFewWaves) {
        const uint32_t from = uniform(r ? end[r - 1] : 0), n = uniform(end[r]) - from;
        if (n == 0) {
            if (!ADD)
                clear_row<Y, false>(row_of_dw<Y>(a, base + r), c - lane * 8, lane, a.cols);
        } else if (n <= kMany) {
            finish<Y, ADD>(a, base + r, c, sum_listed<X>(a, list + from, n, c));
        } else {
            many = 1;
        }
    }
    if (!__syncthreads_or(int(many))) return;
    for (uint32_t r = 0; r < a.run && base + r < a.rows; r++) {
        const uint32_t from = uniform(r ? end[r - 1] : 0), n = uniform(end[r]) - from;
        if (n <= kMany) continue;
        const uint32_t lo = n * wave / kFewWaves, hi = n * (wave + 1) / kFewWaves;
        *reinterpret_cast<f32x8 *>(&part[wave][lane * 8]) = sum_listed<X>(a, list + from + lo, hi - lo, c);
        __syncthreads();
        if (wave == 0) {
            f32x8 sum = *reinterpret_cast<const f32x8 *>(&part[0][lane * 8]);
#pragma unroll
            for (uint32_t w = 1; w < kFewWaves; w++) sum += *reinterpret_cast<const f32x8 *>(&part[w][lane * 8]);
            finish<Y, ADD>(a, base + r, c, sum);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- host

bool bad_tokens(const void *tokens, uint32_t bits, uint64_t n) {
    return (bits != 32 && bits != 64) || n > DF11_EMBEDDING_MAX_TOKENS ||
           (n && (!tokens || !aligned(tokens, bits / 8)));
}

bool bad_matrix(const void *p, uint32_t type, uint64_t stride, uint64_t rows, uint32_t cols) {
    return type > DF11_TYPE_F16 || stride >> 40 || (rows && cols && (!p || !aligned(p, type_bytes(type))));
}

// rows that are written lie apart; those that are read may be one and the same
bool bad_output(const void *p, uint32_t type, uint64_t stride, uint64_t rows, uint32_t cols) {
    return (rows > 1 && stride < cols) || bad_matrix(p, type, stride, rows, cols);
}

// a grid of waves, four a workgroup, holds less than 2^32 threads
bool too_many(uint64_t waves) { return (waves + 3) >> 26; }

// Tokens of a chunk: enough chunks to fill the chip, and no more than their
// borders' sums are worth.
uint32_t chunk_of(uint32_t n) { return n <= 65536 ? 32 : 128; }

// Rows of a sorting workgroup: about 128 workgroups where the table has the rows
// for it, as each reads all tokens; up to 1024, a thread each.
uint32_t run_of(uint32_t rows) {
    uint32_t run = 4;
    while (run < 1024 && (rows + run - 1) / run > 128) run *= 2;
    return run;
}

// Rows of a workgroup of sum_few: some 1024 workgroups.
uint32_t few_run_of(uint32_t rows, uint32_t parts) {
    uint32_t run = 8;
    while (run < kFewRows && uint64_t((rows + run - 1) / run) * parts > 1024) run *= 2;
    return run;
}

uint64_t padded(uint64_t n) { return (n + 31) / 32 * 32; }

// sum_few's calls: a grid of its workgroups holds less than 2^32 threads, and a table
// of 2^26 elements and more is cleared faster beside sum_runs (1000 tokens, 128256 x
// 4096 in float32: 521 us against 400).
bool is_few(uint64_t n, uint64_t rows, uint32_t cols, bool add) {
    const uint32_t parts = (cols + 511) / 512;
    return n <= kFew && (add || rows * cols < 1ull << 26) &&
           (rows + kFewRows - 1) / kFewRows * parts < (1u << 23) - 1;
}

}  // namespace

extern "C" {

int df11_embedding(const df11_embedding_lookup *e, df11_hip_stream stream) {
    if (!e || bad_tokens(e->tokens, e->token_bits, e->n) || e->rows > DF11_EMBEDDING_MAX_ROWS ||
        e->cols > DF11_EMBEDDING_MAX_COLS ||
        bad_matrix(e->table, e->table_type, e->table_stride, e->rows, e->cols) ||
        bad_output(e->out, e->out_type, e->out_stride, e->n, e->cols))
        return DF11_E_INVALID;
    if (!e->n || !e->cols) return DF11_OK;
    LookupArgs a{};
    a.table = e->table, a.tokens = e->tokens, a.out = e->out;
    a.table_stride = e->table_stride, a.out_stride = e->out_stride;
    a.n = uint32_t(e->n), a.rows = uint32_t(e->rows), a.cols = e->cols, a.scale = e->scale;
    a.parts = (e->cols + kPart - 1) / kPart;
    const uint64_t waves = uint64_t(a.n) * a.parts;
    if (too_many(waves)) return DF11_E_INVALID;
    const dim3 grid(uint32_t((waves + 3) / 4));
    hipStream_t st = static_cast<hipStream_t>(stream);
    return with_type(e->table_type, [&](auto t) {
        return with_type(e->out_type, [&](auto y) {
            using T = decltype(t);
            using Y = decltype(y);
            return status(e->token_bits == 64 ? launch(lookup<T, Y, int64_t>, grid, dim3(256), 0, st, a)
                                              : launch(lookup<T, Y, int32_t>, grid, dim3(256), 0, st, a));
        });
    });
}

uint64_t df11_embedding_gradient_scratch_bytes(uint64_t n, uint64_t rows, uint32_t cols) {
    if (n > DF11_EMBEDDING_MAX_TOKENS || rows > DF11_EMBEDDING_MAX_ROWS || cols > DF11_EMBEDDING_MAX_COLS) return 0;
    if (is_few(n, rows, cols, false)) return 0;  // those that add need it less often
    const uint32_t chunk = chunk_of(uint32_t(n));
    return 128 + 16 * padded(n) + 4 * padded(rows) + (n + chunk - 1) / chunk * 2 * 4 * padded(cols);
}

int df11_embedding_gradient(const df11_embedding_grad *g, void *scratch, uint64_t scratch_bytes,
                            df11_hip_stream stream) {
    if (!g || bad_tokens(g->tokens, g->token_bits, g->n) || g->rows > DF11_EMBEDDING_MAX_ROWS ||
        g->cols > DF11_EMBEDDING_MAX_COLS || g->accumulate > 1 ||
        bad_matrix(g->dy, g->dy_type, g->dy_stride, g->n, g->cols) ||
        bad_output(g->dw, g->dw_type, g->dw_stride, g->rows, g->cols))
        return DF11_E_INVALID;
    const bool few = is_few(g->n, g->rows, g->cols, g->accumulate);
    const uint64_t need = few ? 0 : df11_embedding_gradient_scratch_bytes(g->n, g->rows, g->cols);
    if (need && (!scratch || !aligned(scratch, 128) || scratch_bytes < need)) return DF11_E_INVALID;
    if (!g->rows || !g->cols || (!g->n && g->accumulate)) return DF11_OK;
    GradArgs a{};
    a.tokens = g->tokens, a.dy = g->dy, a.dw = g->dw;
    a.dy_stride = g->dy_stride, a.dw_stride = g->dw_stride;
    a.padding = g->padding, a.scale = g->scale;
    a.n = uint32_t(g->n), a.rows = uint32_t(g->rows), a.cols = g->cols;
    a.parts = (a.cols + 511) / 512;
    hipStream_t st = static_cast<hipStream_t>(stream);
    // f(a value of dw's type, one of dy's, one of the tokens')
    const auto with_types = [&](auto f) {
        return with_type(g->dw_type, [&](auto y) {
            return with_type(g->dy_type, [&](auto x) {
                return status(g->token_bits == 64 ? f(y, x, int64_t{}) : f(y, x, int32_t{}));
            });
        });
    };
    if (few) {
        a.run = few_run_of(a.rows, a.parts);
        a.span = uint32_t((g->n + 64 * kFewWaves - 1) / (64 * kFewWaves) * 64);
        const dim3 grid((a.rows + a.run - 1) / a.run * a.parts);
        return with_types([&](auto y, auto x, auto i) {
            using Y = decltype(y);
            using X = decltype(x);
            using I = decltype(i);
            return g->accumulate ? launch(sum_few<X, Y, I, true>, grid, dim3(64 * kFewWaves), 0, st, a)
                                 : launch(sum_few<X, Y, I, false>, grid, dim3(64 * kFewWaves), 0, st, a);
        });
    }
    a.chunk = chunk_of(a.n), a.run = run_of(a.rows);
    a.span = uint32_t((g->n + 64 * kSortWaves - 1) / (64 * kSortWaves) * 64);
    a.kept = static_cast<uint32_t *>(scratch);
    a.sorted = reinterpret_cast<uint4 *>(a.kept + 32);
    a.total = reinterpret_cast<uint32_t *>(a.sorted + padded(a.n));
    a.part = reinterpret_cast<float *>(a.total + padded(a.rows));
    a.part_stride = padded(a.cols);
    const uint32_t chunks = (a.n + a.chunk - 1) / a.chunk;
    const uint64_t joining = uint64_t(chunks) * a.parts, summing = (joining + 3) / 4;
    const uint64_t clearing = g->accumulate ? 0 : ((a.rows + 63) / 64 * uint64_t(a.parts) + 3) / 4;
    if (too_many(4 * std::max(joining, summing + clearing))) return DF11_E_INVALID;
    a.summing = uint32_t(summing);
    const dim3 sorting((a.rows + a.run - 1) / a.run), both(uint32_t(summing + clearing));
    const size_t lds = (kSortWaves + 1) * a.run * 4;
    // dy of the last cache's size, or dw of half of it
    const bool big = g->accumulate ? uint64_t(a.n) * a.cols * type_bytes(g->dy_type) >= 1ull << 28
                                   : uint64_t(a.rows) * a.cols * type_bytes(g->dw_type) >= 1ull << 27;
    int rc = status(g->token_bits == 64 ? launch(sort_tokens<int64_t>, sorting, dim3(64 * kSortWaves), lds, st, a)
                                        : launch(sort_tokens<int32_t>, sorting, dim3(64 * kSortWaves), lds, st, a));
    if (rc != DF11_OK) return rc;
    rc = with_types([&](auto y, auto x, auto) {
        using Y = decltype(y);
        using X = decltype(x);
        if (g->accumulate)
            return big ? launch(sum_runs<X, Y, true, true>, both, dim3(256), 0, st, a)
                       : launch(sum_runs<X, Y, true, false>, both, dim3(256), 0, st, a);
        return big ? launch(sum_runs<X, Y, false, true>, both, dim3(256), 0, st, a)
                   : launch(sum_runs<X, Y, false, false>, both, dim3(256), 0, st, a);
    });
    if (rc != DF11_OK || !joining) return rc;
    return with_type(g->dw_type, [&](auto y) {
        using Y = decltype(y);
        return status(g->accumulate ? launch(join_runs<Y, true>, dim3(uint32_t(joining)), dim3(256), 0, st, a)
                                    : launch(join_runs<Y, false>, dim3(uint32_t(joining)), dim3(256), 0, st, a));
    });
}

}  // extern "C"
