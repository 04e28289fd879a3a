// Products in 8-bit integers: rows quantised to codes with a scale each, and
// the product of activation codes with weight codes on the matrix cores.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "df11.h"
#include "df11_launch.h"

#pragma clang fp contract(off)

namespace {

using df11_detail::launch;

constexpr int kMax = DF11_INT8_MAX_TENSORS;
constexpr uint32_t kThreads = 256;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__bf16 x) { return float(x); }
__device__ __forceinline__ float to_f32(_Float16 x) { return float(x); }

// ---------------------------------------------------------------- quantiser

// 8 elements at any alignment of their type
template <class T>
struct alignas(sizeof(T)) Eight {
    T e[8];
};

// The code of x, as a float: the nearest integer to 127 x / a, ties to even.
//
// 16-bit inputs: t = x inv with inv = 127 / a carries an error of at most
// 2^-23 t.  A quotient of two numbers of 11 bits that is no tie is at least
// 2^-19 t away from one (it is a multiple of 2^-k / 2a where the tie h is about
// 2^-k 127), so rounding t to 21 bits first moves a tie that the error has hidden
// back onto itself and nothing else across one.  p - (p - t) with p = 9 t is
// that rounding.  float32 inputs: the same in float64, 2^-52 against 2^-33,
// rounded to 40 bits.
template <class T>
struct Quotient {
    float pre, inv;
    __device__ explicit Quotient(float a) {
        pre = a < 0x1p-60f ? 0x1p100f : 1.0f;  // keeps 127 / a finite
        inv = 127.0f / (a * pre);
    }
    __device__ float operator()(float x) const {
        const float t = (x * pre) * inv;
        const float p = t * 9.0f;
        return rintf(p - (p - t));
    }
};
template <>
struct Quotient<float> {
    double inv;
    __device__ explicit Quotient(float a) { inv = 127.0 / double(a); }
    __device__ float operator()(float x) const {
        const double t = double(x) * inv;
        const double p = t * 8193.0;
        return float(rint(p - (p - t)));
    }
};

struct QuantArgs {
    const void *src[kMax];
    int8_t *codes[kMax];
    float *scales[kMax];
    uint64_t src_stride[kMax], code_stride[kMax];
    uint32_t cols[kMax];
    uint32_t first[kMax];  // a matrix's first row in the grid; 0xFFFFFFFF past the last
};

// One workgroup per row: the largest magnitude (as bits, so that a NaN or an
// infinity shows), then the codes; the row comes from the caches the second time.
template <class T>
__global__ __launch_bounds__(kThreads) void quantize_rows(QuantArgs a) {
    __shared__ uint32_t top_s[kThreads / 64];
    uint32_t k = 0;
#pragma unroll
    for (int j = 1; j < kMax; j++) k += uint32_t(blockIdx.x >= a.first[j]);
    const uint32_t row = blockIdx.x - a.first[k], cols = a.cols[k];
    const T *x = static_cast<const T *>(a.src[k]) + row * a.src_stride[k];
    int8_t *q = a.codes[k] + row * a.code_stride[k];

    uint32_t top = 0;
    for (uint32_t c = threadIdx.x * 8; c < cols; c += kThreads * 8) {
        if (c + 8 <= cols) {
            const Eight<T> v = *reinterpret_cast<const Eight<T> *>(x + c);
#pragma unroll
            for (int e = 0; e < 8; e++) top = max(top, __float_as_uint(to_f32(v.e[e])) & 0x7FFFFFFFu);
        } else {
            for (uint32_t e = c; e < cols; e++) top = max(top, __float_as_uint(to_f32(x[e])) & 0x7FFFFFFFu);
        }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = max(top, uint32_t(__shfl_xor(int(top), d, 64)));
    if ((threadIdx.x & 63u) == 0) top_s[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(top_s[0], top_s[1]), max(top_s[2], top_s[3]));

    const float amax = __uint_as_float(top);
    const bool bad = top >= 0x7F800000u, zero = bad || top == 0;
    if (threadIdx.x == 0)
        a.scales[k][row] = bad ? __uint_as_float(0x7FC00000u) : amax / 127.0f;
    const Quotient<T> code(zero ? 1.0f : amax);
    for (uint32_t c = threadIdx.x * 8; c < ((cols + 15) & ~15u); c += kThreads * 8) {
        float v[8];
        if (c + 8 <= cols) {
            const Eight<T> e = *reinterpret_cast<const Eight<T> *>(x + c);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = to_f32(e.e[i]);
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 8; i++) v[i] = c + i < cols ? to_f32(x[c + i]) : 0.0f;
        }
        u32x2 out = {0, 0};
        if (!zero) {
#pragma unroll
            for (int i = 0; i < 8; i++) out[i / 4] |= (uint32_t(int(code(v[i]))) & 0xFFu) << (8 * (i % 4));
        }
        *reinterpret_cast<u32x2 *>(q + c) = out;
    }
}

// ---------------------------------------------------------------- product

struct GemmArgs {
    const int8_t *w[kMax];
    const float *w_scale[kMax];
    const int8_t *x[kMax];
    const float *x_scale[kMax];
    void *y[kMax];
    uint64_t y_stride[kMax];
    uint32_t w_stride[kMax], x_stride[kMax];
    uint32_t rows[kMax], cols[kMax];
    uint32_t first[kMax];  // a matrix's first row tile in the grid; 0xFFFFFFFF past the last
    uint32_t n_tokens;
};

// A sum's value in float32.  The compiler would form the last product and its
// F16 rounding in one instruction that rounds once; the empty statement keeps
// the product a float32, so that all three types round the same value.
__device__ __forceinline__ float scaled(int sum, float xs, float ws) {
    float v = (float(sum) * xs) * ws;
    asm("" : "+v"(v));
    return v;
}
template <class Y>
__device__ __forceinline__ void put(Y *y, uint64_t at, int sum, float xs, float ws) {
    y[at] = Y(scaled(sum, xs, ws));
}

// 16 codes of row p at column c of `cols`, zeros past the end
__device__ __forceinline__ i32x4 codes16(const int8_t *p, uint32_t c, uint32_t cols) {
    i32x4 v = {0, 0, 0, 0};
    if (c < cols) v = *reinterpret_cast<const i32x4 *>(p + c);
    return v;
}
// the same with the codes behind `cols` cleared
__device__ __forceinline__ i32x4 codes16_cut(const int8_t *p, uint32_t c, uint32_t cols) {
    i32x4 v = codes16(p, c, cols);
#pragma unroll
    for (uint32_t d = 0; d < 4; d++) {
        const uint32_t at = c + 4 * d;
        const uint32_t keep = at >= cols ? 0u : cols - at;
        if (keep < 4) v[d] = int(uint32_t(v[d]) & ((1u << (8 * keep)) - 1u));
    }
    return v;
}

// Few tokens: a workgroup takes 16 weight rows and NT groups of 16 tokens; its
// four waves split the columns in runs of 256 and their sums meet in LDS.
// Lane 16 q + i of a wave holds row i (or token i) and columns 16 q .. of a
// 16x16x64 product, which the operands' row-major order gives as is.
template <class Y, int NT>
__global__ __launch_bounds__(256) void gemm_rows16(GemmArgs a) {
    __shared__ i32x4 part[3][NT][64];
    uint32_t k = 0;
#pragma unroll
    for (int j = 1; j < kMax; j++) k += uint32_t(blockIdx.x >= a.first[j]);
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t r0 = (blockIdx.x - a.first[k]) * 16, t0 = blockIdx.y * 16 * NT;
    const uint32_t rows = a.rows[k], cols = a.cols[k], i = lane & 15u, q = lane >> 4;
    const int8_t *w = a.w[k] + uint64_t(min(r0 + i, rows - 1)) * a.w_stride[k];
    const int8_t *x[NT];
#pragma unroll
    for (int n = 0; n < NT; n++)
        x[n] = a.x[k] + uint64_t(min(t0 + 16 * n + i, a.n_tokens - 1)) * a.x_stride[k];
    i32x4 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; n++) acc[n] = i32x4{0, 0, 0, 0};
    for (uint32_t c0 = wave * 256; c0 < cols; c0 += 1024) {
        if (c0 + 256 <= cols) {
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const uint32_t c = c0 + 64 * u + 16 * q;
                const i32x4 wv = *reinterpret_cast<const i32x4 *>(w + c);
#pragma unroll
                for (int n = 0; n < NT; n++)
                    acc[n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                        wv, *reinterpret_cast<const i32x4 *>(x[n] + c), acc[n], 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const uint32_t c = c0 + 64 * u + 16 * q;
                const i32x4 wv = codes16_cut(w, c, cols);
#pragma unroll
                for (int n = 0; n < NT; n++)
                    acc[n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, codes16(x[n], c, cols), acc[n],
                                                                   0, 0, 0);
            }
        }
    }
    if (wave) {
#pragma unroll
        for (int n = 0; n < NT; n++) part[wave - 1][n][lane] = acc[n];
    }
    __syncthreads();
    if (wave) return;
    // lane 16 q + j holds rows 4 q .. + 3 of token j
    Y *y = static_cast<Y *>(a.y[k]);
    float ws[4];
#pragma unroll
    for (uint32_t e = 0; e < 4; e++) ws[e] = a.w_scale[k][min(r0 + 4 * q + e, rows - 1)];
#pragma unroll
    for (int n = 0; n < NT; n++) {
        const i32x4 s = acc[n] + part[0][n][lane] + part[1][n][lane] + part[2][n][lane];
        const uint32_t t = t0 + 16 * n + i;
        if (t >= a.n_tokens) continue;
        const float xs = a.x_scale[k][t];
#pragma unroll
        for (uint32_t e = 0; e < 4; e++)
            if (r0 + 4 * q + e < rows) put(y, t * a.y_stride[k] + r0 + 4 * q + e, s[e], xs, ws[e]);
    }
}

// Many tokens: a workgroup computes a tile of BT tokens x BR weight rows, its
// WT x WR waves a part of 32x32 products each.  The tiles' codes go from HBM
// straight to LDS, 128 columns at a time, into one of two buffers while the
// other is multiplied.
//
// A 128-byte row of a tile is 8 chunks of 16 bytes; chunk c of row r lies in
// slot c ^ (r % 8), so that the 8 lanes which LDS serves at once, 8 rows of
// the same chunk, find theirs in 8 different slots.  A lane's load takes the
// chunk that belongs in its slot (LDS receives a wave's lanes in order).
constexpr uint32_t kDepth = 128;  // columns of a stage

typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;

// A tile's rows in global memory: where a lane's chunk lies for each of its
// wave's loads (8 rows a load), relative to the first row.
template <int LOADS>
struct Source {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t at[LOADS];
    __device__ void init(const int8_t *first, uint32_t stride, uint32_t left, uint32_t cols,
                         uint32_t wave, uint32_t lane) {
        const uint32_t last = left - 1;  // rows past the end repeat the last one
        rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(first), 0,
                                                 int(last * stride + ((cols + 15) & ~15u)), 0x00020000);
#pragma unroll
        for (int j = 0; j < LOADS; j++)
            at[j] = min((wave * LOADS + j) * 8 + (lane >> 3), last) * stride;
    }
    // columns c0 .. c0 + 127 to LDS; those of the last stage that lie past
    // the row's last chunk repeat it, so that nothing outside is read
    __device__ void load(int8_t *lds, uint32_t c0, uint32_t cols, uint32_t wave, uint32_t lane) const {
        uint32_t c = 16 * ((lane ^ (lane >> 3)) & 7u);
        if (c0 + kDepth > cols) c = min(c0 + c, (cols - 1) & ~15u) - c0;
#ifdef __HIP_DEVICE_COMPILE__  // the host's pass knows no 16-byte loads to LDS
#pragma unroll
        for (int j = 0; j < LOADS; j++)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (lds_void *)(lds + (wave * LOADS + j) * 1024), 16, at[j] + c, c0, 0, 0);
#endif
    }
};

// Clears the columns from `cols` on of a stage of activations: the weights'
// codes there, whatever they are, then add nothing.
template <int ROWS>
__device__ __forceinline__ void clear_behind(int8_t *lds, uint32_t left, uint32_t threads) {
    for (uint32_t i = threadIdx.x; i < ROWS * 8; i += threads) {
        const uint32_t row = i >> 3, c = 16 * ((i ^ row) & 7u);
        if (c + 16 <= left) continue;
        i32x4 *p = reinterpret_cast<i32x4 *>(lds + i * 16);
        i32x4 v = *p;
#pragma unroll
        for (uint32_t d = 0; d < 4; d++) {
            const uint32_t at = c + 4 * d, keep = at >= left ? 0u : left - at;
            if (keep < 4) v[d] = int(uint32_t(v[d]) & ((1u << (8 * keep)) - 1u));
        }
        *p = v;
    }
}

// A wave's part of a stage: four steps of 32 columns.  The operands of a step
// are read while the one before is multiplied (the scheduling barriers hold
// the reads there).
template <int FT, int FR>
__device__ __forceinline__ void multiply(const int8_t *xs, const int8_t *ws, i32x16 (&acc)[FT][FR]) {
    const uint32_t lane = threadIdx.x & 63u;
    i32x4 x[2][FT], w[2][FR];
    const auto read = [&](uint32_t kk) {
        const uint32_t at = (lane & 31u) * 128 + (((2 * kk + (lane >> 5)) ^ (lane & 7u)) << 4);
#pragma unroll
        for (int f = 0; f < FT; f++) x[kk & 1][f] = *reinterpret_cast<const i32x4 *>(xs + f * 4096 + at);
#pragma unroll
        for (int f = 0; f < FR; f++) w[kk & 1][f] = *reinterpret_cast<const i32x4 *>(ws + f * 4096 + at);
    };
    read(0);
#pragma unroll
    for (uint32_t kk = 0; kk < 4; kk++) {
        if (kk < 3) read(kk + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < FT; f++)
#pragma unroll
            for (int h = 0; h < FR; h++)
                acc[f][h] = __builtin_amdgcn_mfma_i32_32x32x32_i8(x[kk & 1][f], w[kk & 1][h], acc[f][h],
                                                                  0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// This wave's loads have arrived, all waves' reads of the other buffer too.
__device__ __forceinline__ void arrive() {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): loads to LDS are no LDS operations
    __syncthreads();
}

template <class Y, int BT, int BR, int WT, int WR>
__global__ __launch_bounds__(64 * WT * WR) void gemm_tile(GemmArgs a, uint32_t token_tiles,
                                                          uint32_t n_tiles) {
    constexpr int kWaves = WT * WR, FT = BT / WT / 32, FR = BR / WR / 32;
    __shared__ __align__(16) int8_t x0[BT * kDepth], w0[BR * kDepth], x1[BT * kDepth], w1[BR * kDepth];
    // Workgroups go to the 8 XCDs in turn: XCD x takes the x-th run of tiles
    const uint32_t per = n_tiles / 8, rest = n_tiles % 8, xcd = blockIdx.x % 8;
    const uint32_t tile = xcd * per + min(xcd, rest) + blockIdx.x / 8;
    uint32_t k = 0;
#pragma unroll
    for (int j = 1; j < kMax; j++) k += uint32_t(tile >= a.first[j]);
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t rows = a.rows[k], cols = a.cols[k];
    // and walks them 4 token tiles wide, so that the tiles at work on an XCD
    // share both operands in its L2
    const uint32_t row_tiles = (rows + BR - 1) / BR, band = 4 * row_tiles;
    const uint32_t in = tile - a.first[k], t_first = in / band * 4;
    const uint32_t width = min(4u, token_tiles - t_first);
    // (a division by a variable runs on the vector unit)
    const uint32_t r0 = __builtin_amdgcn_readfirstlane((in % band) / width * BR);
    const uint32_t t0 = __builtin_amdgcn_readfirstlane((t_first + (in % band) % width) * BT);

    constexpr int XL = BT / 8 / kWaves, WL = BR / 8 / kWaves;
    Source<XL> sx;
    Source<WL> sw;
    sx.init(a.x[k] + uint64_t(t0) * a.x_stride[k], a.x_stride[k], min(uint32_t(BT), a.n_tokens - t0),
            cols, wave, lane);
    sw.init(a.w[k] + uint64_t(r0) * a.w_stride[k], a.w_stride[k], min(uint32_t(BR), rows - r0), cols,
            wave, lane);
    const uint32_t wt = wave / WR * (BT / WT), wr = wave % WR * (BR / WR);
    i32x16 acc[FT][FR];
#pragma unroll
    for (int f = 0; f < FT; f++)
#pragma unroll
        for (int h = 0; h < FR; h++)
#pragma unroll
            for (int e = 0; e < 16; e++) acc[f][h][e] = 0;

    if (cols) {
        sx.load(x0, 0, cols, wave, lane);
        sw.load(w0, 0, cols, wave, lane);
    }
    uint32_t c = 0;
    for (; c + 2 * kDepth <= cols; c += 2 * kDepth) {
        arrive();
        sx.load(x1, c + kDepth, cols, wave, lane);
        sw.load(w1, c + kDepth, cols, wave, lane);
        multiply<FT, FR>(x0 + wt * kDepth, w0 + wr * kDepth, acc);
        arrive();
        if (c + 2 * kDepth < cols) {
            sx.load(x0, c + 2 * kDepth, cols, wave, lane);
            sw.load(w0, c + 2 * kDepth, cols, wave, lane);
        }
        multiply<FT, FR>(x1 + wt * kDepth, w1 + wr * kDepth, acc);
    }
    if (c < cols) {  // one stage, whole or not, or one whole and one not
        arrive();
        if (c + kDepth < cols) {
            sx.load(x1, c + kDepth, cols, wave, lane);
            sw.load(w1, c + kDepth, cols, wave, lane);
        } else if (cols - c < kDepth) {
            clear_behind<BT>(x0, cols - c, 64 * kWaves);
            __syncthreads();
        }
        multiply<FT, FR>(x0 + wt * kDepth, w0 + wr * kDepth, acc);
        if (c + kDepth < cols) {
            arrive();
            clear_behind<BT>(x1, cols - c - kDepth, 64 * kWaves);
            __syncthreads();
            multiply<FT, FR>(x1 + wt * kDepth, w1 + wr * kDepth, acc);
        }
    }

    // lane l holds row l % 32 of each product, element e token 8 (e / 4) + 4 (l / 32) + e % 4
    Y *y = static_cast<Y *>(a.y[k]);
#pragma unroll
    for (int h = 0; h < FR; h++) {
        const uint32_t r = r0 + wr + 32 * h + (lane & 31u);
        if (r >= rows) continue;
        const float s = a.w_scale[k][r];
#pragma unroll
        for (int f = 0; f < FT; f++) {
#pragma unroll
            for (int e = 0; e < 16; e++) {
                const uint32_t t = t0 + wt + 32 * f + 8 * (e / 4) + 4 * (lane >> 5) + e % 4;
                if (t < a.n_tokens) put(y, t * a.y_stride[k] + r, acc[f][h][e], a.x_scale[k][t], s);
            }
        }
    }
}

// ---------------------------------------------------------------- host

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int status(hipError_t e) { return e == hipSuccess ? DF11_OK : DF11_E_HIP; }

uint32_t type_bytes(uint32_t type) { return type == DF11_TYPE_F32 ? 4 : 2; }

template <class Y, int BT, int BR, int WT, int WR>
int run_tiles(GemmArgs &a, uint32_t n, hipStream_t st) {
    const uint32_t token_tiles = (a.n_tokens + BT - 1) / BT;
    uint64_t tiles = 0;
    for (uint32_t k = 0; k < n; k++) {
        a.first[k] = uint32_t(tiles);
        tiles += uint64_t((a.rows[k] + BR - 1) / BR) * token_tiles;
        if (tiles > 0x7FFFFFFFu) return DF11_E_INVALID;
    }
    return status(launch(gemm_tile<Y, BT, BR, WT, WR>, dim3(uint32_t(tiles)), dim3(64 * WT * WR), 0, st,
                         a, token_tiles, uint32_t(tiles)));
}

template <class Y>
int run_gemm(GemmArgs &a, uint32_t n, hipStream_t st) {
    if (a.n_tokens > 64) return run_tiles<Y, 256, 256, 2, 4>(a, n, st);
    uint32_t tiles = 0;
    for (uint32_t k = 0; k < n; k++) {
        a.first[k] = tiles;
        tiles += (a.rows[k] + 15) / 16;
    }
    const uint32_t t = a.n_tokens;
    if (t <= 16) return status(launch(gemm_rows16<Y, 1>, dim3(tiles), dim3(256), 0, st, a));
    if (t <= 32) return status(launch(gemm_rows16<Y, 2>, dim3(tiles), dim3(256), 0, st, a));
    return status(launch(gemm_rows16<Y, 4>, dim3(tiles, (t + 63) / 64), dim3(256), 0, st, a));
}

}  // namespace

extern "C" {

int df11_quantize_int8(uint32_t src_type, const df11_int8_rows *m, uint32_t n,
                       df11_hip_stream stream) {
    if ((n && !m) || n > kMax || src_type > DF11_TYPE_F16) return DF11_E_INVALID;
    QuantArgs a{};
    uint64_t rows = 0;
    uint32_t used = 0;
    for (uint32_t &f : a.first) f = 0xFFFFFFFFu;
    for (uint32_t k = 0; k < n; k++) {
        const df11_int8_rows &x = m[k];
        if (x.cols > DF11_INT8_MAX_COLS) return DF11_E_INVALID;
        if (!x.rows) continue;
        if (!x.scales || !aligned(x.scales, 4)) return DF11_E_INVALID;
        if (x.cols && (!x.src || !x.codes || !aligned(x.src, type_bytes(src_type)) ||
                       !aligned(x.codes, 16) || x.code_stride % 16 || x.code_stride < x.cols ||
                       x.code_stride > DF11_INT8_MAX_STRIDE ||
                       (x.rows > 1 && x.src_stride < x.cols) || x.src_stride >> 40))
            return DF11_E_INVALID;
        a.src[used] = x.src, a.codes[used] = x.codes, a.scales[used] = x.scales;
        a.src_stride[used] = x.src_stride, a.code_stride[used] = x.code_stride;
        a.cols[used] = x.cols, a.first[used] = uint32_t(rows);
        rows += x.rows;
        used++;
        if (rows > 0x7FFFFFFFu) return DF11_E_INVALID;
    }
    if (!rows) return DF11_OK;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const dim3 grid{uint32_t(rows)};
    switch (src_type) {
    case DF11_TYPE_F32: return status(launch(quantize_rows<float>, grid, dim3(kThreads), 0, st, a));
    case DF11_TYPE_BF16: return status(launch(quantize_rows<__bf16>, grid, dim3(kThreads), 0, st, a));
    default: return status(launch(quantize_rows<_Float16>, grid, dim3(kThreads), 0, st, a));
    }
}

int df11_gemm_int8(uint32_t y_type, const df11_int8_tensor *t, uint32_t n_tensors,
                   uint32_t n_tokens, df11_hip_stream stream) {
    if ((n_tensors && !t) || n_tensors > kMax || y_type > DF11_TYPE_F16) return DF11_E_INVALID;
    if (n_tokens > (1u << 20)) return DF11_E_INVALID;
    GemmArgs a{};
    uint32_t used = 0;
    for (uint32_t &f : a.first) f = 0xFFFFFFFFu;
    for (uint32_t k = 0; k < n_tensors; k++) {
        const df11_int8_tensor &x = t[k];
        if (x.cols > DF11_INT8_MAX_COLS || x.rows > (1u << 24)) return DF11_E_INVALID;
        if (!x.rows || !n_tokens) continue;
        if (!x.w_scale || !x.x_scale || !x.y || !aligned(x.w_scale, 4) || !aligned(x.x_scale, 4) ||
            !aligned(x.y, type_bytes(y_type)) || x.y_stride < x.rows || x.y_stride >> 40)
            return DF11_E_INVALID;
        if (x.cols && (!x.w || !x.x || !aligned(x.w, 16) || !aligned(x.x, 16) || x.w_stride % 16 ||
                       x.x_stride % 16 || x.w_stride < x.cols || x.x_stride < x.cols ||
                       x.w_stride > DF11_INT8_MAX_STRIDE || x.x_stride > DF11_INT8_MAX_STRIDE))
            return DF11_E_INVALID;
        a.w[used] = x.w, a.w_scale[used] = x.w_scale, a.x[used] = x.x, a.x_scale[used] = x.x_scale;
        a.y[used] = x.y, a.y_stride[used] = x.y_stride;
        a.w_stride[used] = uint32_t(x.w_stride), a.x_stride[used] = uint32_t(x.x_stride);
        a.rows[used] = x.rows, a.cols[used] = x.cols;
        used++;
    }
    if (!used) return DF11_OK;
    a.n_tokens = n_tokens;
    hipStream_t st = static_cast<hipStream_t>(stream);
    switch (y_type) {
    case DF11_TYPE_F32: return run_gemm<float>(a, used, st);
    case DF11_TYPE_BF16: return run_gemm<__bf16>(a, used, st);
    default: return run_gemm<_Float16>(a, used, st);
    }
}

}  // extern "C"
