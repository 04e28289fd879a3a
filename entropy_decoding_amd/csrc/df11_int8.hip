// Products in 8-bit integers: rows quantised to codes with a scale each, and
// the product of activation codes with weight codes on the matrix cores.
//
//   y[t][r] = (float(sum_c x[t][c] w[r][c]) * x_scale[t]) * w_scale[r]
//
// The sum is exact in int32, so the result is the same however the columns and
// tiles are split; three forms share the work:
//   linear_one   one token, quantised on the way: workgroups of 16 rows
//   gemm_rows16  up to 16 tokens and few rows: the same on codes
//   gemm_tile    everything else: tiles through LDS, 32 x 64 to 256 x 256
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "df11.h"
#include "df11_launch.h"

#pragma clang fp contract(off)

namespace {

using df11_detail::launch;

constexpr int kMax = DF11_INT8_MAX_TENSORS;

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

// The code of x in the low byte of the result: the nearest integer to 127 x / a,
// ties to even.  A number below 2^22 added to 1.5 2^23 is rounded to an
// integer, whose two's complement is then the low bits.
//
// 16-bit inputs: t = x inv with inv = 127 / a carries an error of at most
// 2^-23 t.  A quotient of two numbers of 11 bits that is no tie is at least
// 2^-19 t away from one (it is a multiple of 2^-k / 2a where the tie h is about
// 2^-k 127), so rounding t to 21 bits first (adding half of the 8 units that
// are then cleared) moves a tie that the error has hidden back onto itself and
// nothing else across one.  float32 inputs: the same in float64, 2^-52 against
// 2^-33, rounded to 40 bits by p - (p - t) with p = 8193 t.
constexpr float kInt = 0x1.8p23f;

template <class T>
struct Quotient {
    float pre, inv;
    __device__ explicit Quotient(float a) {
        pre = a < 0x1p-60f ? 0x1p100f : 1.0f;  // keeps 127 / a finite
        inv = 127.0f / (a * pre);
    }
    template <bool TINY>
    __device__ __forceinline__ uint32_t code(float x) const {
        const float t = (TINY ? x * pre : x) * inv;
        return __float_as_uint(__uint_as_float((__float_as_uint(t) + 4u) & ~7u) + kInt);
    }
    __device__ bool tiny() const { return pre != 1.0f; }
};
template <>
struct Quotient<float> {
    double inv;
    __device__ explicit Quotient(float a) { inv = 127.0 / double(a); }
    template <bool TINY>
    __device__ __forceinline__ uint32_t code(float x) const {
        const double t = double(x) * inv;
        const double p = t * 8193.0;
        return __float_as_uint(float(rint(p - (p - t))) + kInt);
    }
    __device__ bool tiny() const { return false; }
};

// 8 elements at x[c ..], zeros from cols on.  ONCE: they are not wanted again and
// pass the caches by (weights of the 8B block 156 -> 124 us, and their codes
// are still in the caches when they are multiplied; float32's two loads of a
// lane share cache lines, and were slower that way: 199 -> 215 us).
template <bool ONCE, class T>
__device__ __forceinline__ Eight<T> load8(const T *x, uint32_t c, uint32_t cols) {
    typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
    Eight<T> v;
    if (c + 8 <= cols) {
        if constexpr (ONCE && sizeof(T) == 2)
            *reinterpret_cast<u32x4_any *>(&v) =
                __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(x + c));
        else v = *reinterpret_cast<const Eight<T> *>(x + c);
        return v;
    }
#pragma unroll
    for (uint32_t i = 0; i < 8; i++) v.e[i] = c + i < cols ? x[c + i] : T(0.0f);
    return v;
}

// Their largest magnitude, as float32's bits, so that a NaN or an infinity
// shows.  16-bit magnitudes compare as their bits, two at a time.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t top_of(const Eight<float> &v) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; e++) top = max(top, __float_as_uint(v.e[e]) & 0x7FFFFFFFu);
    return top;
}
template <class T>
__device__ __forceinline__ uint32_t top_of(const Eight<T> &v) {
    uint32_t two[4];
    __builtin_memcpy(two, &v, 16);
    u16x2 top = {0, 0};
#pragma unroll
    for (int e = 0; e < 4; e++)
        top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, two[e] & 0x7FFF7FFFu));
    const uint16_t most = max(top[0], top[1]);
    return __float_as_uint(to_f32(__builtin_bit_cast(T, most)));
}

__device__ __forceinline__ uint32_t wave_top(uint32_t top) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = max(top, uint32_t(__shfl_xor(int(top), d, 64)));
    return top;
}

// What a row's largest magnitude says about its codes.
template <class T>
struct Row {
    bool zero;
    float scale;
    Quotient<T> code;
    __device__ explicit Row(uint32_t top)
        : zero(top == 0 || top >= 0x7F800000u),
          scale(top >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(top) / 127.0f),
          code(zero ? 1.0f : __uint_as_float(top)) {}
    template <bool TINY>
    __device__ __forceinline__ u32x2 codes_of(const Eight<T> &v) const {
        u32x2 out;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 4; i++) c[i] = code.template code<TINY>(to_f32(v.e[4 * h + i]));
            out[h] = __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0400u) |
                     __builtin_amdgcn_perm(c[3], c[2], 0x04000C0Cu);
        }
        return out;
    }
    __device__ __forceinline__ u32x2 codes(const Eight<T> &v) const {
        if (zero) return u32x2{0, 0};
        return code.tiny() ? codes_of<true>(v) : codes_of<false>(v);  // the same for the row
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

// One workgroup per row: the largest magnitude, then the codes.  The first kHeld
// times 8 elements of a thread stay in its registers between the two; what a
// longer row has beyond comes from the caches the second time.  Bound by HBM:
// the 8B block's weights take 121 - 126 us from BF16 (5.2 - 5.4 TB/s) and 199 us
// from float32 (5.5 TB/s).  A wave per row (193 us, BF16 then at 158), workgroups
// that stay and load the next row ahead (200 us and more), 512 or 1024 threads
// for rows of 14336 (168 and 256 us against 121) were slower.
constexpr int kHeld = 4;

template <class T, int THREADS>
__global__ __launch_bounds__(THREADS) void quantize_rows(QuantArgs a) {
    __shared__ uint32_t top_s[THREADS / 64];
    uint32_t k = 0;
#pragma unroll
    for (int j = 1; j < kMax; j++) k += uint32_t(blockIdx.x >= a.first[j]);
    const uint32_t r = blockIdx.x - a.first[k], cols = a.cols[k];
    const T *x = static_cast<const T *>(a.src[k]) + r * a.src_stride[k];
    int8_t *q = a.codes[k] + r * a.code_stride[k];
    constexpr uint32_t kPass = THREADS * 8;
    const uint32_t c0 = threadIdx.x * 8, end = (cols + 15) & ~15u;
    Eight<T> held[kHeld];
    uint32_t top = 0;
#pragma unroll
    for (int n = 0; n < kHeld; n++)
        if (c0 + n * kPass < cols) held[n] = load8<true>(x, c0 + n * kPass, cols);
#pragma unroll
    for (int n = 0; n < kHeld; n++)
        if (c0 + n * kPass < cols) top = max(top, top_of(held[n]));
    for (uint32_t c = c0 + kHeld * kPass; c < cols; c += kPass) top = max(top, top_of(load8<false>(x, c, cols)));
    top = wave_top(top);
    if ((threadIdx.x & 63u) == 0) top_s[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int p = 0; p < THREADS / 64; p++) top = max(top, top_s[p]);
    const Row<T> row(top);
    if (threadIdx.x == 0) a.scales[k][r] = row.scale;
#pragma unroll
    for (int n = 0; n < kHeld; n++) {
        const uint32_t c = c0 + n * kPass;
        if (c < cols) *reinterpret_cast<u32x2 *>(q + c) = row.codes(held[n]);
        else if (c < end) *reinterpret_cast<u32x2 *>(q + c) = u32x2{0, 0};
    }
    for (uint32_t c = c0 + kHeld * kPass; c < end; c += kPass)
        *reinterpret_cast<u32x2 *>(q + c) = row.codes(load8<true>(x, c, cols));
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
// 16 codes of a row at column c, those behind `cols` cleared; only the row is read
__device__ __forceinline__ i32x4 codes16(const int8_t *p, uint32_t c, uint32_t cols) {
    i32x4 v = *reinterpret_cast<const i32x4 *>(p + min(c, (cols - 1) & ~15u));
#pragma unroll
    for (uint32_t d = 0; d < 4; d++) {
        const uint32_t at = c + 4 * d, keep = at >= cols ? 0u : cols - at;
        if (keep < 4) v[d] = int(uint32_t(v[d]) & ((1u << (8 * keep)) - 1u));
    }
    return v;
}

// Few rows and at most 16 tokens, where what counts is the time of one
// workgroup: it takes 16 weight rows, its eight waves split the columns in runs
// of 128, and each has the weights of 512 columns in flight at once.  The
// waves' sums meet in LDS.  Lane 16 q + i of a wave holds row i (or token i) and
// columns 16 q .. of a 16x16x64 product, which the operands' row-major order
// gives as is.
constexpr uint32_t kRowWaves = 8;
constexpr uint32_t kRun = kRowWaves * 128;

// The next operands of a wave, from column c0 on (c0 - 16 q is the same in all
// its lanes): four runs, or what is left of one; returns how many products.
struct Runs {
    i32x4 w[8];
    int n;
    __device__ __forceinline__ void load(const int8_t *p, uint32_t c0, uint32_t base, uint32_t cols) {
        if (base + 3 * kRun + 128 <= cols) {
            n = 8;
#pragma unroll
            for (int u = 0; u < 8; u++)
                w[u] = *reinterpret_cast<const i32x4 *>(p + c0 + kRun * (u / 2) + 64 * (u % 2));
        } else if (base < cols) {
            n = 2;
#pragma unroll
            for (int u = 0; u < 2; u++) w[u] = codes16(p, c0 + 64 * u, cols);
        } else {
            n = 0;
        }
    }
};

// The product of the workgroup's rows; x(c) gives a lane 16 activation codes at
// column c < cols rounded up to 16.  `runs` holds the first operands.
template <class X>
__device__ __forceinline__ i32x4 rows16_sum(Runs &runs, const int8_t *w, uint32_t c0, uint32_t base,
                                            uint32_t cols, X x) {
    i32x4 acc = {0, 0, 0, 0};
    const uint32_t last = (cols - 1) & ~15u;
    while (runs.n) {
        Runs next;  // on their way while these are multiplied
        const uint32_t step = runs.n == 8 ? 4 * kRun : kRun;
        next.load(w, c0 + step, base + step, cols);
        if (runs.n == 8) {
            i32x4 xv[8];
#pragma unroll
            for (int u = 0; u < 8; u++) xv[u] = x(c0 + kRun * (u / 2) + 64 * (u % 2));
#pragma unroll
            for (int u = 0; u < 8; u++)
                acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(runs.w[u], xv[u], acc, 0, 0, 0);
        } else {
#pragma unroll
            for (int u = 0; u < 2; u++)
                acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(runs.w[u], x(min(c0 + 64 * u, last)), acc,
                                                            0, 0, 0);
        }
        runs = next;
        c0 += step, base += step;
    }
    return acc;
}

// Adds the waves' sums and stores: lane 16 q + j holds rows 4 q .. + 3 of token j.
template <class Y>
__device__ __forceinline__ void rows16_store(i32x4 acc, i32x4 (*part)[64], uint32_t wave, uint32_t lane,
                                             Y *y, uint32_t rows_left, bool token, float xs,
                                             const float *ws) {
    if (wave) part[wave - 1][lane] = acc;
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (uint32_t p = 0; p < kRowWaves - 1; p++) acc += part[p][lane];
    const uint32_t q = lane >> 4;
#pragma unroll
    for (uint32_t e = 0; e < 4; e++)
        if (token && 4 * q + e < rows_left) y[4 * q + e] = Y(scaled(acc[e], xs, ws[e]));
}

template <class Y>
__global__ __launch_bounds__(64 * kRowWaves) void gemm_rows16(GemmArgs a) {
    __shared__ i32x4 part[kRowWaves - 1][64];
    uint32_t k = 0;
#pragma unroll
    for (int j = 1; j < kMax; j++) k += uint32_t(blockIdx.x >= a.first[j]);
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r0 = (blockIdx.x - a.first[k]) * 16;
    const uint32_t rows = a.rows[k], cols = a.cols[k], i = lane & 15u, q = lane >> 4;
    const int8_t *w = a.w[k] + uint64_t(min(r0 + i, rows - 1)) * a.w_stride[k];
    const uint32_t token = min(i, a.n_tokens - 1);
    const int8_t *x = a.x[k] + uint64_t(token) * a.x_stride[k];
    Runs runs;
    runs.load(w, wave * 128 + 16 * q, wave * 128, cols);
    const float xs = a.x_scale[k][token];
    float ws[4];
#pragma unroll
    for (uint32_t e = 0; e < 4; e++) ws[e] = a.w_scale[k][min(r0 + 4 * q + e, rows - 1)];
    const i32x4 acc = rows16_sum(runs, w, wave * 128 + 16 * q, wave * 128, cols, [&](uint32_t c) {
        return *reinterpret_cast<const i32x4 *>(x + c);
    });
    rows16_store(acc, part, wave, lane, static_cast<Y *>(a.y[k]) + i * a.y_stride[k] + r0, rows - r0,
                 i < a.n_tokens, xs, ws);
}

// One token that is not quantised yet: every workgroup quantises it for itself
// while its first weights are on their way, which spares the launch before.
// Bound by reading the weights: 46.3 us on the 8B block (4.7 TB/s) and 156 us on
// the 70B block (5.5 TB/s), 4.5 us on 1024 x 1024, against 55.2, 165 and 7.2 us
// with a launch for the codes before.  Holding the kernel to 80 or 64 registers
// for more waves made it slower (8B block 59 and 79 us): its loads in flight
// need them.
constexpr uint32_t kOneMaxCols = 32768;  // the codes' room in LDS

template <class X, class Y>
__global__ __launch_bounds__(64 * kRowWaves) void linear_one(GemmArgs a) {
    __shared__ i32x4 part[kRowWaves - 1][64];
    __shared__ uint32_t top_s[kRowWaves];
    extern __shared__ __align__(16) int8_t codes[];
    uint32_t k = 0;
#pragma unroll
    for (int j = 1; j < kMax; j++) k += uint32_t(blockIdx.x >= a.first[j]);
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r0 = (blockIdx.x - a.first[k]) * 16;
    const uint32_t rows = a.rows[k], cols = a.cols[k], i = lane & 15u, q = lane >> 4;
    const int8_t *w = a.w[k] + uint64_t(min(r0 + i, rows - 1)) * a.w_stride[k];
    const X *x = reinterpret_cast<const X *>(a.x[k]);
    Runs runs;
    runs.load(w, wave * 128 + 16 * q, wave * 128, cols);
    float ws[4];
#pragma unroll
    for (uint32_t e = 0; e < 4; e++) ws[e] = a.w_scale[k][min(r0 + 4 * q + e, rows - 1)];

    constexpr uint32_t kStep = 64 * kRowWaves * 8;
    const uint32_t own = threadIdx.x * 8;  // a thread's first elements, held for their codes
    const Eight<X> held = load8<false>(x, own, cols);
    uint32_t top = top_of(held);
    for (uint32_t c = own + kStep; c < cols; c += kStep) top = max(top, top_of(load8<false>(x, c, cols)));
    top = wave_top(top);
    if (lane == 0) top_s[wave] = top;
    __syncthreads();
#pragma unroll
    for (uint32_t p = 0; p < kRowWaves; p++) top = max(top, top_s[p]);
    const Row<X> row(top);
    if (own < ((cols + 15) & ~15u)) *reinterpret_cast<u32x2 *>(codes + own) = row.codes(held);
    for (uint32_t c = own + kStep; c < ((cols + 15) & ~15u); c += kStep)
        *reinterpret_cast<u32x2 *>(codes + c) = row.codes(load8<false>(x, c, cols));
    __syncthreads();

    const i32x4 acc = rows16_sum(runs, w, wave * 128 + 16 * q, wave * 128, cols, [&](uint32_t c) {
        return *reinterpret_cast<const i32x4 *>(codes + c);
    });
    rows16_store(acc, part, wave, lane, static_cast<Y *>(a.y[k]) + r0, rows - r0, i == 0, row.scale, ws);
}

// More tokens: a workgroup computes a tile of BT tokens x BR weight rows, its
// WT x WR waves a part each, of 16x16x64 products (these draw less power than
// 32x32x32 ones: alone, with random codes, they run at 3.67 POP/s against 3.44,
// both held back by the power limit; the kernel gained 5%).  The tiles' codes go from HBM straight to LDS, 128 columns
// (a stage) at a time, into one of NB buffers, NB - 1 stages ahead of the
// products, so that a workgroup has up to 60 KB on its way.
//
// What bounds it: up to 64 tokens the reading of the weights (8B block, 32
// tokens: 54 us, 4.1 TB/s, the 70B block 161 us, 5.4 TB/s); between, the L2's
// throughput (12 - 17 TB/s into LDS, the larger tile the fewer bytes); from
// some 1000 tokens on the products' power (70B block, 4096 tokens: 2.65 ms,
// 2.65 POP/s).  Not kept for 256 x 256: four waves of 128 x 128 instead of
// eight (2.27 against 2.40 POP/s, then), stages of 64 columns in four buffers
// (2.31 against 2.45), touching the next stages' lines ahead (2.05 against 2.23).
//
// A 128-byte row of a tile is 8 chunks of 16 bytes; chunk c of row r lies in
// slot c ^ (r / 2 % 8): LDS serves 16 lanes of a 16-byte read at once, and
// these find the same chunk of their rows without a conflict (4.1 cycles a
// read, as for consecutive addresses; 8.1 with r % 8, 32 without a swizzle).
// A lane's load takes the chunk that belongs in its slot (LDS receives a
// wave's lanes in order).
constexpr uint32_t kDepth = 128;  // columns of a stage

typedef __attribute__((address_space(3))) void lds_void;

// A tile's rows in global memory: where a lane's chunk lies for each of its
// wave's loads (8 rows a load), relative to the first row.
template <int LOADS>
struct Source {
    int8_t *first;
    uint32_t bytes, at[LOADS];
    // lane's first column in load j: the chunk of its slot
    static __device__ uint32_t column(uint32_t wave, uint32_t lane, int j) {
        return 16 * ((lane ^ (((wave * LOADS + j) * 8 + (lane >> 3)) >> 1)) & 7u);
    }
    __device__ void init(const int8_t *p, uint32_t stride, uint32_t left, uint32_t cols,
                         uint32_t wave, uint32_t lane) {
        const uint32_t last = left - 1;  // rows past the end repeat the last one
        first = const_cast<int8_t *>(p);
        bytes = last * stride + ((cols + 15) & ~15u);
#pragma unroll
        for (int j = 0; j < LOADS; j++)
            at[j] = min((wave * LOADS + j) * 8 + (lane >> 3), last) * stride + column(wave, lane, j);
    }
    // columns tail .. `cols` to LDS; chunks past a row's last one repeat it, so
    // that nothing outside is read
    __device__ __forceinline__ void load_tail(int8_t *lds, uint32_t tail, uint32_t cols, uint32_t wave,
                                              uint32_t lane) const {
        Source s = *this;
#pragma unroll
        for (int j = 0; j < LOADS; j++) {
            const uint32_t c = column(wave, lane, j);
            s.at[j] -= c - (min(tail + c, (cols - 1) & ~15u) - tail);
        }
        s.load(lds, tail, true, wave);
    }
    // columns c0 .. c0 + 127 to LDS, loads `from` .. `to`; zeros if not `on`
    __device__ __forceinline__ void load(int8_t *lds, uint32_t c0, bool on, uint32_t wave,
                                         int from = 0, int to = LOADS) const {
#ifdef __HIP_DEVICE_COMPILE__  // the host's pass knows no 16-byte loads to LDS
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc(first, 0, on ? int(bytes) : 0, 0x00020000);
#pragma unroll
        for (int j = 0; j < LOADS; j++)
            if (j >= from && j < to)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rsrc, (lds_void *)(lds + (wave * LOADS + j) * 1024), 16, at[j], c0, 0, 0);
#endif
    }
};

// Clears the columns from `cols` on of a stage of activations: the weights'
// codes there, whatever they are, then add nothing.
template <int ROWS>
__device__ __forceinline__ void clear_behind(int8_t *lds, uint32_t left, uint32_t threads) {
    for (uint32_t i = threadIdx.x; i < ROWS * 8; i += threads) {
        const uint32_t row = i >> 3, c = 16 * ((i ^ (row >> 1)) & 7u);
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

// The operands of one step of 64 columns.
template <int FT, int FR>
struct Operands {
    i32x4 x[FT], w[FR];
};

template <class Y, int BT, int BR, int WT, int WR, int NB>
__global__ __launch_bounds__(64 * WT * WR) void gemm_tile(GemmArgs a, uint32_t token_tiles) {
    constexpr int kWaves = WT * WR, FT = BT / WT / 16, FR = BR / WR / 16;
    // a buffer is an object of its own, so that the compiler sees that reads
    // of one do not wait for loads to another
    __shared__ __align__(16) int8_t x0[BT * kDepth], w0[BR * kDepth], x1[BT * kDepth], w1[BR * kDepth];
    __shared__ __align__(16) int8_t x2[NB > 2 ? BT * kDepth : 16], w2[NB > 2 ? BR * kDepth : 16];
    __shared__ __align__(16) int8_t x3[NB > 3 ? BT * kDepth : 16], w3[NB > 3 ? BR * kDepth : 16];
    __shared__ __align__(16) int8_t x4[NB > 4 ? BT * kDepth : 16], w4[NB > 4 ? BR * kDepth : 16];
    __shared__ __align__(16) int8_t x5[NB > 4 ? BT * kDepth : 16], w5[NB > 4 ? BR * kDepth : 16];
    __shared__ __align__(16) float w_scale[BR];
    // Workgroups go to the 8 XCDs in turn: every XCD takes one run of a
    // matrix's tiles (first counts an XCD's tiles, so that matrices of longer
    // rows burden all of them alike)
    const uint32_t turn = blockIdx.x / 8;
    uint32_t k = 0;
#pragma unroll
    for (int j = 1; j < kMax; j++) k += uint32_t(turn >= a.first[j]);
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t rows = a.rows[k], cols = a.cols[k];
    const uint32_t row_tiles = (rows + BR - 1) / BR, band = 4 * row_tiles;
    const uint32_t tiles = row_tiles * token_tiles;
    const uint32_t in = blockIdx.x % 8 * ((tiles + 7) / 8) + turn - a.first[k];
    if (in >= tiles) return;
    // and walks them 4 token tiles wide, so that the tiles at work on an XCD
    // share both operands in its L2
    const uint32_t t_first = in / band * 4;
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
    for (uint32_t r = threadIdx.x; r < BR; r += 64 * kWaves)
        w_scale[r] = a.w_scale[k][min(r0 + r, rows - 1)];
    i32x4 acc[FT][FR];
#pragma unroll
    for (int f = 0; f < FT; f++)
#pragma unroll
        for (int h = 0; h < FR; h++)
#pragma unroll
            for (int e = 0; e < 4; e++) acc[f][h][e] = 0;

    // A step of 64 columns multiplies one set of operands while the next set
    // is read from LDS; before a stage's last step its waves meet: the next
    // stage has arrived then, and this one's buffer is free for the one after
    // it, whose loads go out between the products of that step.  The
    // scheduling barriers hold the reads and loads between the products.
    Operands<FT, FR> even, odd;
    const auto read = [&](Operands<FT, FR> &o, const int8_t *xs, const int8_t *ws, uint32_t kk, int f) {
        const uint32_t at = (lane & 15u) * 128 + (((4 * kk + (lane >> 4)) ^ (lane >> 1 & 7u)) << 4);
        if (f < FT) o.x[f] = *reinterpret_cast<const i32x4 *>(xs + wt * kDepth + f * 2048 + at);
        if (f < FR) o.w[f] = *reinterpret_cast<const i32x4 *>(ws + wr * kDepth + f * 2048 + at);
    };
    constexpr int kF = FT > FR ? FT : FR;
    const auto products = [&](const Operands<FT, FR> &o, int f) {
        __builtin_amdgcn_sched_barrier(0);
        if (f < FT) {
#pragma unroll
            for (int h = 0; h < FR; h++)
                acc[f][h] = __builtin_amdgcn_mfma_i32_16x16x64_i8(o.w[h], o.x[f], acc[f][h], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    // the next stage has arrived when at most the loads of the NB - 2 behind it are out
    constexpr int kOut = (NB - 2) * (XL + WL);
    static_assert(kOut < 64, "the counter of loads");
    const auto arrived = [&] {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((kOut & 15) | (kOut >> 4 << 14) | 0x0070);  // and lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // Stage 0 is the last 1 .. 128 columns, cleared behind the end; stage s > 0
    // starts at column 128 (s - 1).  Loads for stages past the last give zeros,
    // so that the loop has no conditions and the stages that fill up a round
    // of the buffers add nothing.
    const uint32_t stages = (cols + kDepth - 1) / kDepth;
    const auto stage = [&](int8_t *xs, int8_t *ws, int8_t *xn, int8_t *wn, uint32_t s) {
#pragma unroll
        for (int f = 0; f < kF; f++) {
            read(odd, xs, ws, 1, f);
            products(even, f);
        }
        arrived();
        const bool on = s + NB < stages;
#pragma unroll
        for (int f = 0; f < kF; f++) {
            sx.load(xs, (s + NB - 1) * kDepth, on, wave, f * XL / kF, (f + 1) * XL / kF);
            sw.load(ws, (s + NB - 1) * kDepth, on, wave, f * WL / kF, (f + 1) * WL / kF);
            read(even, xn, wn, 0, f);
            products(odd, f);
        }
    };
    if (cols) {
        const uint32_t tail = (stages - 1) * kDepth;
        sx.load_tail(x0, tail, cols, wave, lane);
        sw.load_tail(w0, tail, cols, wave, lane);
        __builtin_amdgcn_sched_barrier(0);
        const auto begin = [&](int8_t *xs, int8_t *ws, uint32_t s) {
            sx.load(xs, (s - 1) * kDepth, s < stages, wave);
            sw.load(ws, (s - 1) * kDepth, s < stages, wave);
            __builtin_amdgcn_sched_barrier(0);
        };
        begin(x1, w1, 1);
        if constexpr (NB > 2) begin(x2, w2, 2);
        if constexpr (NB > 3) begin(x3, w3, 3);
        if constexpr (NB > 4) begin(x4, w4, 4), begin(x5, w5, 5);
        constexpr int kFirst = (NB - 1) * (XL + WL);
        static_assert(kFirst < 64, "the counter of loads");
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((kFirst & 15) | (kFirst >> 4 << 14) | 0x0070);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (cols % kDepth) {
            clear_behind<BT>(x0, cols - tail, 64 * kWaves);
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        }
#pragma unroll
        for (int f = 0; f < kF; f++) read(even, x0, w0, 0, f);
        for (uint32_t s = 0; s < stages; s += NB) {
            stage(x0, w0, x1, w1, s);
            if constexpr (NB == 2) {
                stage(x1, w1, x0, w0, s + 1);
            } else if constexpr (NB == 3) {
                stage(x1, w1, x2, w2, s + 1);
                stage(x2, w2, x0, w0, s + 2);
            } else if constexpr (NB == 4) {
                stage(x1, w1, x2, w2, s + 1);
                stage(x2, w2, x3, w3, s + 2);
                stage(x3, w3, x0, w0, s + 3);
            } else {
                static_assert(NB == 6, "2, 3, 4 or 6 buffers");
                stage(x1, w1, x2, w2, s + 1);
                stage(x2, w2, x3, w3, s + 2);
                stage(x3, w3, x4, w4, s + 3);
                stage(x4, w4, x5, w5, s + 4);
                stage(x5, w5, x0, w0, s + 5);
            }
        }
    }

    // Lane l holds token l % 16 and rows 4 (l / 16) .. + 3 of each product.  The
    // results pass through LDS (the stages' buffers are
    // free once the last loads, of zeros, have come), 128 bytes of each of 32
    // tokens at a time, so that a token's rows leave in whole cache lines.
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
    __syncthreads();
    constexpr int kRows = std::min<int>(128 / sizeof(Y), 16 * FR), kParts = kRows / 16;
    constexpr uint32_t kBytes = kRows * sizeof(Y), kPitch = kBytes + 16;  // tokens in different banks
    constexpr uint32_t kX = BT * kDepth / (32 * kPitch), kW = BR * kDepth / (32 * kPitch);
    static_assert(FR % kParts == 0, "whole rows of results");
    constexpr bool kOwn = kWaves > int(2 * kX + kW);  // small buffers: memory of its own
    __shared__ __align__(16) int8_t results[kOwn ? kWaves * 32 * kPitch : 16];
    int8_t *out = kOwn ? results + wave * (32 * kPitch)
                       : (wave < kX ? x0 : wave < 2 * kX ? x1 : w0) +
                             (wave < 2 * kX ? wave % std::max(kX, 1u) : wave - 2 * kX) * (32 * kPitch);
    Y *y = static_cast<Y *>(a.y[k]);
    typedef Y Y4 __attribute__((ext_vector_type(4)));
    typedef Y Y16B __attribute__((ext_vector_type(16 / sizeof(Y))));
    typedef Y16B Y16B_any __attribute__((aligned(sizeof(Y))));
    float xs[FT];
#pragma unroll
    for (int f = 0; f < FT; f++)
        xs[f] = a.x_scale[k][min(t0 + wt + 16 * f + (lane & 15u), a.n_tokens - 1)];
#pragma unroll
    for (int f = 0; f < FT / 2; f++) {
#pragma unroll
        for (int h0 = 0; h0 < FR; h0 += kParts) {
#pragma unroll
            for (int h = h0; h < h0 + kParts; h++) {
                const uint32_t r = 4 * (lane >> 4);
                const float4 ws = *reinterpret_cast<const float4 *>(&w_scale[wr + 16 * h + r]);
#pragma unroll
                for (int g = 0; g < 2; g++) {
                    Y4 v;
#pragma unroll
                    for (int e = 0; e < 4; e++) v[e] = Y(scaled(acc[2 * f + g][h][e], xs[2 * f + g], (&ws.x)[e]));
                    *reinterpret_cast<Y4 *>(out + (16 * g + (lane & 15u)) * kPitch +
                                            (16 * (h - h0) + r) * sizeof(Y)) = v;
                }
            }
            // a wave's LDS operations take effect in order: no barrier
            constexpr uint32_t kLanes = kBytes / 16;  // of a token
            const uint32_t chunk = lane % kLanes, r = r0 + wr + 16 * h0 + chunk * (16 / sizeof(Y));
#pragma unroll
            for (uint32_t p = 0; p < kLanes / 2; p++) {
                const uint32_t i = 64 / kLanes * p + lane / kLanes, tok = t0 + wt + 32 * f + i;
                const Y16B v = *reinterpret_cast<const Y16B *>(out + i * kPitch + chunk * 16);
                if (tok >= a.n_tokens) continue;
                Y *to = y + tok * a.y_stride[k] + r;
                if (r + 16 / sizeof(Y) <= rows) {
                    // results of many tokens pass the caches by, which keeps the
                    // weights there (8B block, 512 tokens: 115 against 127 us)
                    if constexpr (BT >= 128)
                        __builtin_nontemporal_store(Y16B_any(v), reinterpret_cast<Y16B_any *>(to));
                    else *reinterpret_cast<Y16B_any *>(to) = v;
                } else {
#pragma unroll
                    for (uint32_t e = 0; e < 16 / sizeof(Y) - 1; e++)
                        if (r + e < rows) to[e] = v[e];
                }
            }
        }
    }
}

// ---------------------------------------------------------------- host

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int status(hipError_t e) { return e == hipSuccess ? DF11_OK : DF11_E_HIP; }

// a grid holds less than 2^32 threads
bool too_many(uint64_t groups, uint32_t threads) { return groups * threads >> 32; }

// Few long rows: 1024 threads each, so that a row's time counts less (3 rows of
// 28058: 28 -> 26 us for the whole of quantiser and product).
template <class T>
int run_rows(const QuantArgs &a, uint32_t rows, uint32_t longest, hipStream_t st) {
    if (rows <= 512 && longest > 2048)
        return status(launch(quantize_rows<T, 1024>, dim3(rows), dim3(1024), 0, st, a));
    return status(launch(quantize_rows<T, 256>, dim3(rows), dim3(256), 0, st, a));
}

// Rows that start on a cache line: a stage's 128 columns are then one line of a
// row and not parts of two (8B block, 128 tokens: 52 us, against 69 with rows
// 64 bytes and 73 with rows 16 bytes off).
uint64_t code_stride(uint64_t cols) { return (cols + 127) / 128 * 128; }
uint64_t scale_bytes(uint64_t rows) { return (rows * 4 + 127) / 128 * 128; }

uint32_t type_bytes(uint32_t type) { return type == DF11_TYPE_F32 ? 4 : 2; }

template <class Y, int BT, int BR, int WT, int WR, int NB>
int run_tiles(GemmArgs &a, uint32_t n, hipStream_t st) {
    const uint32_t token_tiles = (a.n_tokens + BT - 1) / BT;
    uint64_t turns = 0;
    for (uint32_t k = 0; k < n; k++) {
        a.first[k] = uint32_t(turns);
        turns += (uint64_t((a.rows[k] + BR - 1) / BR) * token_tiles + 7) / 8;
        if (too_many(turns * 8, 64 * WT * WR)) return DF11_E_INVALID;
    }
    return status(launch(gemm_tile<Y, BT, BR, WT, WR, NB>, dim3(uint32_t(turns) * 8), dim3(64 * WT * WR), 0,
                         st, a, token_tiles));
}

// How long tiles of bt tokens x br rows take, in microseconds: all compute units
// together, or the longest tile alone (stages of 128 columns; 3 more for a
// tile's start and end).
float tiles_time(const GemmArgs &a, uint32_t n, uint32_t bt, uint32_t br, float busy, float alone) {
    const uint64_t token_tiles = (a.n_tokens + bt - 1) / bt;
    uint64_t stages = 0;
    uint32_t longest = 0;
    for (uint32_t k = 0; k < n; k++) {
        const uint32_t s = (a.cols[k] + kDepth - 1) / kDepth + 3;
        stages += (a.rows[k] + br - 1) / br * token_tiles * s;
        longest = std::max(longest, s);
    }
    return std::max(float(stages) / 256 * busy, float(longest) * alone);
}

// first of workgroups of 16 rows; returns their number
uint32_t sixteens(GemmArgs &a, uint32_t n) {
    uint32_t tiles = 0;
    for (uint32_t k = 0; k < n; k++) {
        a.first[k] = tiles;
        tiles += (a.rows[k] + 15) / 16;
    }
    return tiles;
}

template <class X, class Y>
int run_one(GemmArgs &a, uint32_t n, hipStream_t st) {
    uint32_t cols = 0;
    for (uint32_t k = 0; k < n; k++) cols = std::max(cols, a.cols[k]);
    const uint32_t tiles = sixteens(a, n);
    if (too_many(tiles, 64 * kRowWaves)) return DF11_E_INVALID;
    return status(launch(linear_one<X, Y>, dim3(tiles), dim3(64 * kRowWaves), (cols + 15) & ~15u, st, a));
}

template <class X>
int run_one(uint32_t y_type, GemmArgs &a, uint32_t n, hipStream_t st) {
    switch (y_type) {
    case DF11_TYPE_F32: return run_one<X, float>(a, n, st);
    case DF11_TYPE_BF16: return run_one<X, __bf16>(a, n, st);
    default: return run_one<X, _Float16>(a, n, st);
    }
}

template <class Y>
int run_gemm(GemmArgs &a, uint32_t n, hipStream_t st) {
    if (a.n_tokens <= 32) {
        // Workgroups of 16 rows are the faster form for one token, and up to 16
        // where they are no more than the compute units (4096 x 4096: 7.2 us
        // against 9.6 with 1 token, 8.4 against 10.4 with 16); more of them
        // read too much of the activations (8B block: 43.4 against 48.0 us
        // with 1 token, but 48.4 against 48.6 with 4 and 66 against 51 with 16).
        const uint32_t tiles = sixteens(a, n);
        if ((a.n_tokens == 1 && !too_many(tiles, 64 * kRowWaves)) || (a.n_tokens <= 16 && tiles <= 256))
            return status(launch(gemm_rows16<Y>, dim3(tiles), dim3(64 * kRowWaves), 0, st, a));
        return run_tiles<Y, 32, 64, 1, 2, 6>(a, n, st);
    }
    // The tile with the least time by tiles_time, whose rates (per stage, with the
    // chip full and with one tile alone) were fitted to the times of every tile
    // on the 8B and the 70B block and on 4096 x 4096 and 8192 x 8192, 64 to 2048
    // tokens: of those 40 the rule misses the best by 4% once and by 1% twice.
    // What it decides (8B block, us, tiles of 64 / 128 / 256 x 128 / 256): 128
    // tokens 50 / 58 / 78 / 127, 256 tokens 94 / 77 / 110 / 168, 512 tokens
    // 192 / 141 / 126 / 189, 2048 tokens 816 / 540 / 437 / 416.
    const float t64 = tiles_time(a, n, 64, 64, 0.20f, 0.23f);
    const float t128 = tiles_time(a, n, 128, 128, 0.63f, 0.42f);
    const float t256x128 = tiles_time(a, n, 256, 128, 0.89f, 0.93f);
    const float t256 = tiles_time(a, n, 256, 256, 1.47f, 1.47f);
    const float least = std::min(std::min(t64, t128), std::min(t256x128, t256));
    if (least == t64) return run_tiles<Y, 64, 64, 2, 2, 4>(a, n, st);
    if (least == t128) return run_tiles<Y, 128, 128, 4, 2, 4>(a, n, st);
    if (least == t256x128) return run_tiles<Y, 256, 128, 4, 2, 3>(a, n, st);
    return run_tiles<Y, 256, 256, 2, 4, 2>(a, n, st);
}

// Checks the product's arguments and fills the kernels' (used: the matrices with
// work).  x_align: 16 for codes, an element's bytes for one token's values,
// which have neither scales nor a stride.
int prepare_gemm(uint32_t y_type, const df11_int8_tensor *t, uint32_t n_tensors, uint32_t n_tokens,
                 uint32_t x_align, GemmArgs &a, uint32_t &used) {
    const bool codes = x_align == 16;
    if ((n_tensors && !t) || n_tensors > kMax || y_type > DF11_TYPE_F16) return DF11_E_INVALID;
    if (n_tokens > (1u << 20)) return DF11_E_INVALID;
    uint32_t order[kMax];
    for (uint32_t &f : a.first) f = 0xFFFFFFFFu;
    // the matrices of the longest rows first, so that the last workgroups are short ones
    for (uint32_t k = 0; k < n_tensors; k++) order[k] = k;
    std::stable_sort(order, order + n_tensors,
                     [t](uint32_t i, uint32_t j) { return t[i].cols > t[j].cols; });
    for (uint32_t k = 0; k < n_tensors; k++) {
        const df11_int8_tensor &x = t[order[k]];
        if (x.cols > DF11_INT8_MAX_COLS || x.rows > (1u << 24)) return DF11_E_INVALID;
        if (!x.rows || !n_tokens) continue;
        if (!x.w_scale || !x.y || !aligned(x.w_scale, 4) || !aligned(x.y, type_bytes(y_type)) ||
            x.y_stride < x.rows || x.y_stride >> 40 ||
            (codes && (!x.x_scale || !aligned(x.x_scale, 4))))
            return DF11_E_INVALID;
        if (x.cols && (!x.w || !x.x || !aligned(x.w, 16) || !aligned(x.x, x_align) || x.w_stride % 16 ||
                       x.w_stride < x.cols || x.w_stride > DF11_INT8_MAX_STRIDE ||
                       (codes && (x.x_stride % 16 || x.x_stride < x.cols ||
                                  x.x_stride > DF11_INT8_MAX_STRIDE))))
            return DF11_E_INVALID;
        a.w[used] = x.w, a.w_scale[used] = x.w_scale, a.x[used] = x.x, a.x_scale[used] = x.x_scale;
        a.y[used] = x.y, a.y_stride[used] = x.y_stride;
        a.w_stride[used] = uint32_t(x.w_stride), a.x_stride[used] = uint32_t(x.x_stride);
        a.rows[used] = x.rows, a.cols[used] = x.cols;
        used++;
    }
    a.n_tokens = n_tokens;
    return DF11_OK;
}

// linear_one's calls
bool one_token(const df11_int8_tensor *t, uint32_t n, uint32_t n_tokens) {
    bool one = n && n_tokens == 1;
    for (uint32_t k = 0; one && k < n; k++) one = t[k].cols >= 1 && t[k].cols <= kOneMaxCols;
    return one;
}

int launch_gemm(uint32_t y_type, GemmArgs &a, uint32_t used, hipStream_t st) {
    switch (y_type) {
    case DF11_TYPE_F32: return run_gemm<float>(a, used, st);
    case DF11_TYPE_BF16: return run_gemm<__bf16>(a, used, st);
    default: return run_gemm<_Float16>(a, used, st);
    }
}

}  // namespace

extern "C" {

int df11_quantize_int8(uint32_t src_type, const df11_int8_rows *m, uint32_t n,
                       df11_hip_stream stream) {
    if ((n && !m) || n > kMax || src_type > DF11_TYPE_F16) return DF11_E_INVALID;
    QuantArgs a{};
    uint64_t rows = 0;
    uint32_t used = 0, longest = 0;
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
        longest = std::max(longest, x.cols);
        rows += x.rows;
        used++;
        if (too_many(rows, 256)) return DF11_E_INVALID;
    }
    if (!rows) return DF11_OK;
    hipStream_t st = static_cast<hipStream_t>(stream);
    switch (src_type) {
    case DF11_TYPE_F32: return run_rows<float>(a, uint32_t(rows), longest, st);
    case DF11_TYPE_BF16: return run_rows<__bf16>(a, uint32_t(rows), longest, st);
    default: return run_rows<_Float16>(a, uint32_t(rows), longest, st);
    }
}

int df11_gemm_int8(uint32_t y_type, const df11_int8_tensor *t, uint32_t n_tensors,
                   uint32_t n_tokens, df11_hip_stream stream) {
    GemmArgs a{};
    uint32_t used = 0;
    const int rc = prepare_gemm(y_type, t, n_tensors, n_tokens, 16, a, used);
    return rc == DF11_OK && used ? launch_gemm(y_type, a, used, static_cast<hipStream_t>(stream)) : rc;
}

uint64_t df11_linear_int8_scratch_bytes(const df11_int8_tensor *t, uint32_t n_tensors,
                                        uint32_t n_tokens) {
    if (!t || one_token(t, n_tensors, n_tokens)) return 0;
    uint64_t bytes = 0;
    for (uint32_t k = 0; k < n_tensors; k++)
        bytes += n_tokens * code_stride(t[k].cols) + scale_bytes(n_tokens);
    return bytes;
}

int df11_linear_int8(uint32_t x_type, uint32_t y_type, const df11_int8_tensor *t,
                     uint32_t n_tensors, uint32_t n_tokens, void *scratch, uint64_t scratch_bytes,
                     df11_hip_stream stream) {
    if ((n_tensors && !t) || n_tensors > kMax || n_tokens > (1u << 20) || x_type > DF11_TYPE_F16)
        return DF11_E_INVALID;
    const uint64_t need = df11_linear_int8_scratch_bytes(t, n_tensors, n_tokens);
    if (!aligned(scratch, 16) || scratch_bytes < need || (need && !scratch)) return DF11_E_INVALID;
    hipStream_t st = static_cast<hipStream_t>(stream);
    GemmArgs a{};
    uint32_t used = 0;
    if (one_token(t, n_tensors, n_tokens)) {
        const int rc = prepare_gemm(y_type, t, n_tensors, n_tokens, type_bytes(x_type), a, used);
        if (rc != DF11_OK || !used) return rc;
        switch (x_type) {
        case DF11_TYPE_F32: return run_one<float>(y_type, a, used, st);
        case DF11_TYPE_BF16: return run_one<__bf16>(y_type, a, used, st);
        default: return run_one<_Float16>(y_type, a, used, st);
        }
    }
    df11_int8_rows rows[kMax];
    df11_int8_tensor q[kMax];
    uint32_t n_rows = 0;
    int8_t *at = static_cast<int8_t *>(scratch);
    for (uint32_t k = 0; k < n_tensors; k++) {
        if (t[k].cols > DF11_INT8_MAX_COLS) return DF11_E_INVALID;
        uint32_t j = 0;
        while (j < n_rows && (rows[j].src != t[k].x || rows[j].src_stride != t[k].x_stride ||
                              rows[j].cols != t[k].cols))
            j++;
        if (j == n_rows) {
            df11_int8_rows &r = rows[n_rows++];
            r.src = t[k].x, r.src_stride = t[k].x_stride;
            r.rows = n_tokens, r.cols = t[k].cols;
            r.code_stride = code_stride(r.cols);
            r.codes = at;
            at += n_tokens * r.code_stride;
            r.scales = reinterpret_cast<float *>(at);
            at += scale_bytes(n_tokens);
        }
        q[k] = t[k];
        q[k].x = rows[j].codes, q[k].x_scale = rows[j].scales, q[k].x_stride = rows[j].code_stride;
    }
    // the product's arguments are checked before the first launch
    int rc = prepare_gemm(y_type, q, n_tensors, n_tokens, 16, a, used);
    if (rc == DF11_OK) rc = df11_quantize_int8(x_type, rows, n_rows, stream);
    return rc == DF11_OK && used ? launch_gemm(y_type, a, used, st) : rc;
}

}  // extern "C"
