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
// sorted rows, where each one's run ends, and sums of runs that cross chunks.
struct GradArgs {
    const void *tokens, *dy;
    void *dw;
    uint32_t *kept, *order, *row, *end;
    float *part;
    uint64_t dy_stride, dw_stride, part_stride;
    int64_t padding;
    uint32_t n, rows, cols, span, run, parts, chunk;
    float scale;
};

constexpr uint32_t kSortWaves = 16;

// Sorts the tokens by row, stably, in one launch without a word between its
// workgroups: each owns `run` neighbouring rows, reads all tokens twice, and
// keeps those of its rows.  The first reading counts them by wave and row, and
// all tokens of earlier rows, which says where its rows begin; the second puts
// each at its place.  A wave reads `span` consecutive tokens, in order, so
// places within a row ascend with the position.  With ZERO the rows without a
// token are cleared on the way.
template <class I, class Y, bool ZERO>
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
    constexpr uint32_t kLoads = 8;
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
        total[threadIdx.x] = mine ? upto : 0;  // where the row's run ends; 0: no token
        uint32_t at = upto - mine;
        for (uint32_t w = 0; w < kSortWaves; w++) {
            const uint32_t c = count[w * a.run + threadIdx.x];
            count[w * a.run + threadIdx.x] = at;
            at += c;
        }
        if (blockIdx.x == gridDim.x - 1 && threadIdx.x == a.run - 1) *a.kept = upto;
    }
    __syncthreads();

    if constexpr (ZERO) {
        for (uint32_t r = wave; r < a.run && base + r < a.rows; r += kSortWaves) {
            if (total[r]) continue;
            Y *row = static_cast<Y *>(a.dw) + (base + r) * a.dw_stride;
            for (uint32_t c = lane * 8; c < a.cols; c += 512) store_group<Y>(row, c, a.cols, f32x8(0.0f));
        }
    }

    // A wave's places are its own: its LDS operations take effect in order.
    volatile uint32_t *place = count + wave * a.run;
    for (uint32_t p = from; p < to; p += 64 * kLoads) {
        read(p, row);
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

// Sums the runs of equal rows within chunks of sorted tokens, a wave for a
// chunk's 512 columns.  A run that crosses into another chunk leaves its sum of
// this one in the chunk's first (it began before) or second slot.
template <class X, class Y, bool ADD>
__global__ __launch_bounds__(256) void sum_runs(GradArgs a) {
    const uint32_t wave = uniform(blockIdx.x * 4 + (threadIdx.x >> 6)), lane = threadIdx.x & 63u;
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

// Rows of a sorting workgroup: at least as many workgroups as compute units
// where the table has the rows for it; up to 1024, a thread each.
uint32_t run_of(uint32_t rows) {
    uint32_t run = 4;
    while (run < 1024 && (rows + run - 1) / run > 512) run *= 2;
    return run;
}

uint64_t padded(uint64_t n) { return (n + 31) / 32 * 32; }

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

uint64_t df11_embedding_gradient_scratch_bytes(uint64_t n, uint32_t cols) {
    if (n > DF11_EMBEDDING_MAX_TOKENS || cols > DF11_EMBEDDING_MAX_COLS) return 0;
    const uint32_t chunk = chunk_of(uint32_t(n));
    return 128 + 3 * 4 * padded(n) + (n + chunk - 1) / chunk * 2 * 4 * padded(cols);
}

int df11_embedding_gradient(const df11_embedding_grad *g, void *scratch, uint64_t scratch_bytes,
                            df11_hip_stream stream) {
    if (!g || bad_tokens(g->tokens, g->token_bits, g->n) || g->rows > DF11_EMBEDDING_MAX_ROWS ||
        g->cols > DF11_EMBEDDING_MAX_COLS || g->accumulate > 1 ||
        bad_matrix(g->dy, g->dy_type, g->dy_stride, g->n, g->cols) ||
        bad_output(g->dw, g->dw_type, g->dw_stride, g->rows, g->cols))
        return DF11_E_INVALID;
    if (!scratch || !aligned(scratch, 128) ||
        scratch_bytes < df11_embedding_gradient_scratch_bytes(g->n, g->cols))
        return DF11_E_INVALID;
    if (!g->rows || !g->cols || (!g->n && g->accumulate)) return DF11_OK;
    GradArgs a{};
    a.tokens = g->tokens, a.dy = g->dy, a.dw = g->dw;
    a.dy_stride = g->dy_stride, a.dw_stride = g->dw_stride;
    a.padding = g->padding, a.scale = g->scale;
    a.n = uint32_t(g->n), a.rows = uint32_t(g->rows), a.cols = g->cols;
    a.chunk = chunk_of(a.n), a.run = run_of(a.rows), a.parts = (a.cols + 511) / 512;
    a.span = uint32_t((g->n + 64 * kSortWaves - 1) / (64 * kSortWaves) * 64);
    a.kept = static_cast<uint32_t *>(scratch);
    a.order = a.kept + 32, a.row = a.order + padded(a.n), a.end = a.row + padded(a.n);
    a.part = reinterpret_cast<float *>(a.end + padded(a.n));
    a.part_stride = padded(a.cols);
    const uint32_t chunks = (a.n + a.chunk - 1) / a.chunk;
    const uint64_t waves = uint64_t(chunks) * a.parts;
    if (too_many(waves)) return DF11_E_INVALID;
    const dim3 sorting((a.rows + a.run - 1) / a.run), summing(uint32_t((waves + 3) / 4));
    const size_t lds = (kSortWaves + 1) * a.run * 4;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return with_type(g->dw_type, [&](auto y) {
        using Y = decltype(y);
        const auto sort = [&](auto i) {
            using I = decltype(i);
            return g->accumulate ? launch(sort_tokens<I, Y, false>, sorting, dim3(64 * kSortWaves), lds, st, a)
                                 : launch(sort_tokens<I, Y, true>, sorting, dim3(64 * kSortWaves), lds, st, a);
        };
        int rc = status(g->token_bits == 64 ? sort(int64_t{}) : sort(int32_t{}));
        if (rc != DF11_OK || !a.n) return rc;
        rc = with_type(g->dy_type, [&](auto x) {
            using X = decltype(x);
            return status(g->accumulate ? launch(sum_runs<X, Y, true>, summing, dim3(256), 0, st, a)
                                        : launch(sum_runs<X, Y, false>, summing, dim3(256), 0, st, a));
        });
        if (rc != DF11_OK || chunks < 2) return rc;
        return status(g->accumulate ? launch(join_runs<Y, true>, summing, dim3(256), 0, st, a)
                                    : launch(join_runs<Y, false>, summing, dim3(256), 0, st, a));
    });
}

}  // extern "C"
