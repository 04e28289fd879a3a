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

__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

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

// What the launches hand on: positions of the kept tokens sorted by row, the
// sorted rows, where each one's run ends (by sorted token, and by row of the
// table: 0 where there is none), and sums of runs that cross chunks.
struct GradArgs {
    const void *tokens, *dy;
    void *dw;
    uint32_t *kept, *order, *row, *end, *total;
    float *part;
    uint64_t dy_stride, dw_stride, part_stride;
    int64_t padding;
    uint32_t n, rows, cols, span, run, parts, chunk;
    uint32_t summing;  // workgroups that sum; those behind them clear rows
    float scale;
};

constexpr uint32_t kSortWaves = 16;

// Sorts the tokens by row, stably, in one launch without a word between its
// workgroups: each owns `run` neighbouring rows, reads all tokens twice, and
// keeps those of its rows.  The first reading counts them by wave and row, and
// all tokens of earlier rows, which says where its rows begin; the second puts
// each at its place.  A wave reads `span` consecutive tokens, in order, so
// places within a row ascend with the position.  What bounds it is the reading
// of all tokens by all workgroups, and its latency; up to 32768 tokens are held in
// registers in between (TIME_SORT us of them, 34 us reading twice).
template <class I>
__global__ __launch_bounds__(64 * kSortWaves) void sort_tokens(GradArgs a) {
    extern __shared__ uint32_t shared[];
    uint32_t *count = shared, *total = shared + kSortWaves * a.run;  // [wave][row], [row]
    __shared__ uint32_t sums[kSortWaves];
    const uint32_t lane = threadIdx.x & 63u, wave = uniform(threadIdx.x >> 6);
    const uint32_t base = blockIdx.x * a.run;
    for (uint32_t i = threadIdx.x; i < kSortWaves * a.run; i += 64 * kSortWaves) count[i] = 0;
    __syncthreads();

    const uint32_t from = min(a.n, wave * a.span), to = min(a.n, from + a.span);
    const I *tokens = static_cast<const I *>(a.tokens);
    constexpr uint32_t kLoads = 32;
    // the row of each of a wave's next tokens, 2^32 - 1 for those that are not kept
    const auto read = [&](uint32_t p, uint32_t (&row)[kLoads]) {
        I t[kLoads];
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++) {
            const uint32_t i = p + 64 * u + lane;
            t[u] = i < to ? tokens[i] : I(-1);
        }
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++)
            row[u] = int64_t(t[u]) == a.padding ? 0xFFFFFFFFu : row_of(t[u], a.rows);
    };
    uint32_t below = 0, row[kLoads];
    for (uint32_t p = from; p < to; p += 64 * kLoads) {
        read(p, row);
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++) {
            below += uint32_t(row[u] < base);
            const uint32_t r = row[u] - base;
            if (row[u] >= base && r < a.run) atomicAdd(&count[wave * a.run + r], 1u);
        }
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) below += __shfl_xor(below, d);
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
        total[threadIdx.x] = mine ? upto : 0;
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

    // A wave's places are its own: its LDS operations take effect in order.
    volatile uint32_t *place = count + wave * a.run;
    for (uint32_t p = from; p < to; p += 64 * kLoads) {
        if (a.span > 64 * kLoads) read(p, row);  // or they are held from the first reading
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++) {
            const uint32_t r = row[u] - base;
            const bool in = row[u] >= base && r < a.run && row[u] != 0xFFFFFFFFu;
            for (uint64_t left = __ballot(in); left;) {
                const uint32_t first = __builtin_ctzll(left);
                const uint32_t r0 = __builtin_amdgcn_readlane(r, first);
                const uint64_t same = __ballot(in && r == r0);
                const uint32_t at = place[r0];
                if (in && r == r0) {
                    const uint32_t to_place = at + __popcll(same & ((1ull << lane) - 1));
                    a.order[to_place] = p + 64 * u + lane;
                    a.row[to_place] = row[u];
                    a.end[to_place] = total[r0];
                }
                if (lane == first) place[r0] = at + __popcll(same);
                left &= ~same;
            }
        }
    }
}

template <class Y>
__device__ __forceinline__ void finish(const GradArgs &a, uint32_t row, uint32_t c, f32x8 sum, bool add) {
    Y *dw = static_cast<Y *>(a.dw) + row * a.dw_stride;
    sum = scaled(sum, a.scale);
    if (add) sum += widen<Y>(load_group<Y>(dw, c, a.cols));
    store_group<Y>(dw, c, a.cols, sum);
}

// Clears the rows without a token among 64 rows, 512 columns of them.
template <class Y>
__device__ __forceinline__ void clear_rows(const GradArgs &a, uint32_t wave, uint32_t lane) {
    const uint32_t first = wave / a.parts * 64, c = wave % a.parts * 512 + lane * 8;
    const uint32_t row = first + lane;
    for (uint64_t none = __ballot(row < a.rows && a.total[min(row, a.rows - 1)] == 0); none; none &= none - 1)
        store_group<Y>(static_cast<Y *>(a.dw) + (first + __builtin_ctzll(none)) * a.dw_stride, c, a.cols, f32x8(0.0f));
}

// Sums the runs of equal rows within chunks of sorted tokens, a wave for a
// chunk's 512 columns.  A run that crosses into another chunk leaves its sum of
// this one in the chunk's first (it began before) or second slot.  Without ADD
// further workgroups clear the rows without a token meanwhile.  Bound by HBM.
template <class X, class Y, bool ADD>
__global__ __launch_bounds__(256) void sum_runs(GradArgs a) {
    const uint32_t lane = threadIdx.x & 63u;
    if (!ADD && blockIdx.x >= a.summing)
        return clear_rows<Y>(a, uniform((blockIdx.x - a.summing) * 4 + (threadIdx.x >> 6)), lane);
    const uint32_t wave = uniform(blockIdx.x * 4 + (threadIdx.x >> 6));
    const uint32_t chunk = wave / a.parts, c = wave % a.parts * 512 + lane * 8;
    const uint32_t kept = *a.kept, from = chunk * a.chunk;
    if (from >= kept) return;
    const uint32_t to = min(kept, from + a.chunk);
    const X *dy = static_cast<const X *>(a.dy);
    const bool began_before = from && a.row[from - 1] == a.row[from];
    constexpr uint32_t kLoads = 8;
    f32x8 sum = 0.0f;
    uint32_t first = from;  // of the run
    for (uint32_t j = from; j < to; j += kLoads) {
        typename Group<X>::type v[kLoads];
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++)
            v[u] = load_group<X>(dy + a.order[min(j + u, to - 1)] * a.dy_stride, c, a.cols);
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++) {
            if (j + u >= to) break;
            sum += widen<X>(v[u]);
            const uint32_t end = a.end[j + u];
            if (j + u + 1 < to && j + u + 1 != end) continue;
            // the run's last token here
            const bool before = first == from && began_before;
            if (before || end > to) {
                float *part = a.part + (2 * uint64_t(chunk) + (before ? 0 : 1)) * a.part_stride + c;
                if (c < a.cols) *reinterpret_cast<f32x8 *>(part) = sum;
            } else {
                finish<Y>(a, a.row[j + u], c, sum, ADD);
            }
            sum = 0.0f;
            first = j + u + 1;
        }
    }
}

// Joins the sums of a run that begins in this chunk and goes on in others.
template <class Y, bool ADD>
__global__ __launch_bounds__(256) void join_runs(GradArgs a) {
    const uint32_t wave = uniform(blockIdx.x * 4 + (threadIdx.x >> 6)), lane = threadIdx.x & 63u;
    const uint32_t chunk = wave / a.parts, c = wave % a.parts * 512 + lane * 8;
    const uint32_t kept = *a.kept, from = chunk * a.chunk;
    if (from >= kept || kept - from <= a.chunk) return;
    const uint32_t last = from + a.chunk - 1, row = a.row[last], end = a.end[last];
    if (end <= from + a.chunk) return;                                       // ends here
    if (from && a.row[from] == row && a.row[from - 1] == row) return;  // began before
    if (c >= a.cols) return;
    const uint32_t chunks = (end - 1) / a.chunk - chunk;  // behind this one
    const float *part = a.part + (2 * uint64_t(chunk) + 1) * a.part_stride + c;
    f32x8 sum = *reinterpret_cast<const f32x8 *>(part);
    part += a.part_stride;
    constexpr uint32_t kLoads = 4;
    for (uint32_t k = 0; k < chunks; k += kLoads) {
        f32x8 v[kLoads];
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++)
            v[u] = *reinterpret_cast<const f32x8 *>(part + 2 * uint64_t(min(k + u, chunks - 1)) * a.part_stride);
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++)
            if (k + u < chunks) sum += v[u];
    }
    finish<Y>(a, row, c, sum, ADD);
}

// Few tokens: all of it in one launch.  A workgroup owns `run` neighbouring rows
// and 512 columns of them, sorts its rows' tokens in LDS and sums them; a row of
// many tokens is shared by its waves.  2048 tokens are 4 for each of its threads,
// which hold them in registers.  300 tokens, 1999 x 513: TIME_SMALL us on the GPU
// where the three launches above take 18.
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
#pragma unroll
    for (uint32_t u = 0; u < kFewEach; u++)
        if (row[u] != 0xFFFFFFFFu) atomicAdd(&count[wave][row[u]], 1u);
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
    volatile uint32_t *place = count[wave];
#pragma unroll
    for (uint32_t u = 0; u < kFewEach; u++) {
        for (uint64_t left = __ballot(row[u] != 0xFFFFFFFFu); left;) {
            const uint32_t first = __builtin_ctzll(left);
            const uint32_t r0 = __builtin_amdgcn_readlane(row[u], first);
            const uint64_t same = __ballot(row[u] == r0);
            const uint32_t at = place[r0];
            if (row[u] == r0) list[at + __popcll(same & ((1ull << lane) - 1))] = uint16_t(wave * a.span + 64 * u + lane);
            if (lane == first) place[r0] = at + __popcll(same);
            left &= ~same;
        }
    }
    __syncthreads();

    uint64_t many = 0;  // whether a row of many tokens is among the workgroup's
    for (uint32_t r = wave; r < a.run && base + r < a.rows; r += kFewWaves) {
        const uint32_t from = uniform(r ? end[r - 1] : 0), n = uniform(end[r]) - from;
        if (n == 0) {
            if (!ADD) store_group<Y>(static_cast<Y *>(a.dw) + (base + r) * a.dw_stride, c, a.cols, f32x8(0.0f));
        } else if (n <= kMany) {
            finish<Y>(a, base + r, c, sum_listed<X>(a, list + from, n, c), ADD);
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
            finish<Y>(a, base + r, c, sum, ADD);
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
uint32_t chunk_of(uint32_t n) { return n <= 4096 ? 16 : n <= 65536 ? 32 : 128; }

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

// sum_few's calls (a grid of its workgroups holds less than 2^32 threads)
bool is_few(uint64_t n, uint64_t rows, uint32_t cols) {
    const uint32_t parts = (cols + 511) / 512;
    return n <= kFew && (rows + kFewRows - 1) / kFewRows * parts < (1u << 23) - 1;
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
    if (is_few(n, rows, cols)) return 0;
    const uint32_t chunk = chunk_of(uint32_t(n));
    return 128 + 4 * (3 * padded(n) + padded(rows)) + (n + chunk - 1) / chunk * 2 * 4 * padded(cols);
}

int df11_embedding_gradient(const df11_embedding_grad *g, void *scratch, uint64_t scratch_bytes,
                            df11_hip_stream stream) {
    if (!g || bad_tokens(g->tokens, g->token_bits, g->n) || g->rows > DF11_EMBEDDING_MAX_ROWS ||
        g->cols > DF11_EMBEDDING_MAX_COLS || g->accumulate > 1 ||
        bad_matrix(g->dy, g->dy_type, g->dy_stride, g->n, g->cols) ||
        bad_output(g->dw, g->dw_type, g->dw_stride, g->rows, g->cols))
        return DF11_E_INVALID;
    const uint64_t need = df11_embedding_gradient_scratch_bytes(g->n, g->rows, g->cols);
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
    if (is_few(g->n, g->rows, g->cols)) {
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
    a.order = a.kept + 32, a.row = a.order + padded(a.n), a.end = a.row + padded(a.n);
    a.total = a.end + padded(a.n);
    a.part = reinterpret_cast<float *>(a.total + padded(a.rows));
    a.part_stride = padded(a.cols);
    const uint32_t chunks = (a.n + a.chunk - 1) / a.chunk;
    const uint64_t summing = (uint64_t(chunks) * a.parts + 3) / 4;
    const uint64_t clearing = g->accumulate ? 0 : ((a.rows + 63) / 64 * uint64_t(a.parts) + 3) / 4;
    if (too_many(4 * (summing + clearing))) return DF11_E_INVALID;
    a.summing = uint32_t(summing);
    const dim3 sorting((a.rows + a.run - 1) / a.run), both(uint32_t(summing + clearing));
    const size_t lds = (kSortWaves + 1) * a.run * 4;
    int rc = status(g->token_bits == 64 ? launch(sort_tokens<int64_t>, sorting, dim3(64 * kSortWaves), lds, st, a)
                                        : launch(sort_tokens<int32_t>, sorting, dim3(64 * kSortWaves), lds, st, a));
    if (rc != DF11_OK) return rc;
    rc = with_types([&](auto y, auto x, auto) {
        using Y = decltype(y);
        using X = decltype(x);
        return g->accumulate ? launch(sum_runs<X, Y, true>, both, dim3(256), 0, st, a)
                             : launch(sum_runs<X, Y, false>, both, dim3(256), 0, st, a);
    });
    if (rc != DF11_OK) return rc;
    return with_type(g->dw_type, [&](auto y) {
        using Y = decltype(y);
        return status(g->accumulate ? launch(join_runs<Y, true>, dim3(a.summing), dim3(256), 0, st, a)
                                    : launch(join_runs<Y, false>, dim3(a.summing), dim3(256), 0, st, a));
    });
}

}  // extern "C"
