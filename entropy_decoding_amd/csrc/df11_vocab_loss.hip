// Softmax cross entropy of hidden states under an output head, without keeping
// the logits, and its gradients.
//
//   l[t][v] = x[t] . w[v]      lse[t] = log(sum_v exp l[t][v])      loss[t] = lse[t] - l[t][target t]
//   g[t][v] = p_t exp(l[t][v] - lse[t]) - q_t [v = target t]        dx = s g w        dw = s g^T x
//
// where p_t and q_t come from the gradients of loss and lse, divided by s, their
// digits.  All four products (the logits twice) run on one kernel of tiles on the
// matrix cores, with the logits' two uses in its epilogues: a tile of logits leaves its
// rows' largest value and sum of exponentials, or its part of g.  g exists in BF16 for
// a piece of the vocabulary at a time.
//
//   stats tiles     logits of a tile; the target's, and the others' largest value and sum
//   loss_join       joins tiles and pieces: lse and loss
//   pick, gather    the tokens that have a gradient, one behind the other (up to 1024
//                   tokens in one launch)
//   grad tiles      logits again; g
//   dx tiles        g w, added up over pieces in float32
//   dw tiles        s g^T x
//   spread          dx of all tokens, times s
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "df11.h"
#include "df11_elements.h"
#include "df11_launch.h"

#pragma clang fp contract(off)

namespace {

using namespace df11_detail;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

// What the tiles of a launch compute.
enum Kind { STATS, GRAD, DX, DW, DW_PAST };  // DW_PAST: DW stored past the caches

constexpr uint32_t kDepth = 64;  // of a stage: columns (or rows) that are summed over
constexpr uint32_t kNever = 0x7FFFFF00u;  // an offset behind every buffer: the load gives zeros

// The tiles, their threads, how many workgroups a compute unit holds, and the
// microseconds of a stage with the chip full of them and with one of them alone,
// fitted to the logits of 16 to 8192 tokens x 128256 rows x 4096 columns and of
// 1001 x 32003 x 1000.  Of 70 other shapes (1 to 8192 tokens, 1000 to 131072 rows, 64 to
// 8192 columns, at random) the tile chosen, with each of the six in its place, cost the
// call 1.6% of the best one's time in the median for the logits, 23% at most (one or
// two tokens, or some 100 under few columns: up to 25 us); for g 1% and 15%, for dx 1%
// and 6%, for dw nothing and 5%.
struct Tile {
    uint32_t t, r, threads, held;
    float full, alone;
};
constexpr Tile kTiles[] = {{32, 64, 128, 2, 0.30f, 0.20f},   {64, 64, 256, 2, 0.42f, 0.23f},
                           {64, 128, 256, 2, 0.73f, 0.35f},  {128, 128, 512, 1, 0.57f, 0.42f},
                           {256, 128, 512, 1, 0.95f, 0.8f},  {256, 256, 512, 1, 1.49f, 1.3f}};

constexpr uint32_t held(int t, int r) {
    for (const Tile &tile : kTiles)
        if (int(tile.t) == t && int(tile.r) == r) return tile.held;
    return 0;
}

// A product y[t][r] = sum over k of a[t][k] b[r][k].  The operands of DX and
// DW that hold k as rows are read transposed: b of DX (w), a and b of DW (g, x).
struct TileArgs {
    const __bf16 *a, *b;
    uint64_t a_stride, b_stride;
    const uint32_t *count;  // where not null, the number of tokens (t, or k of DW)
    uint32_t t_size, r_size, k_size;
    // g in one to three terms, each `a_term` elements behind the one before; the stages
    // go over k once for each
    uint32_t terms;
    uint64_t a_term;
    uint32_t splits, split_stages;  // of k
    // STATS and GRAD
    const void *targets;
    uint32_t target_bits, first;
    float2 *part;         // [token / 16][tile][token % 16]: largest, sum of the others
    uint32_t part_tiles;
    float *told;          // the targets' logits
    const float *lse;
    const float2 *factor; // p, and q or (exact_target) what g is at the target
    uint32_t exact_target;
    const uint32_t *target_of;
    __bf16 *g;
    uint64_t g_stride, g_term;
    uint32_t r_padded;  // g is zero up to there
    // DX and DW
    const float *scale;   // of DW
    void *y;
    uint64_t y_stride, y_split;
    uint32_t add;
};

// A tile's operand whose rows are consecutive in k: 128 bytes of each of ROWS
// rows.  They are 8 chunks of 16 bytes; chunk c of row r lies in slot
// c ^ (r / 2 % 8), which serves the 16-byte reads of 16 rows without a bank
// conflict.  A lane's load takes the chunk that belongs in its slot (LDS
// receives a wave's lanes in order).
template <int ROWS, int WAVES>
struct Straight {
    static constexpr int kLoads = ROWS / 8 / WAVES;
    const char *base;
    uint32_t bytes, at[kLoads];
    static __device__ uint32_t column(uint32_t wave, uint32_t lane, int j) {
        return 8 * ((lane ^ (((wave * kLoads + j) * 8 + (lane >> 3)) >> 1)) & 7u);
    }
    // rows from `p` on, `left` of them (at least one); rows past the end repeat the last
    __device__ void init(const __bf16 *p, uint64_t stride, uint32_t left, uint32_t cols, uint32_t wave,
                         uint32_t lane) {
        const uint32_t last = min(left, uint32_t(ROWS)) - 1;
        base = reinterpret_cast<const char *>(p);
        bytes = (last * uint32_t(stride) + cols) * 2;
#pragma unroll
        for (int j = 0; j < kLoads; j++)
            at[j] = (min((wave * kLoads + j) * 8 + (lane >> 3), last) * uint32_t(stride) +
                     column(wave, lane, j)) * 2;
    }
    // columns k0 .. k0 + 63 (of the term `behind` elements on) to LDS; zeros if not
    // `on`, and for columns from `left` on
    template <bool TAIL = false>
    __device__ __forceinline__ void load(char *lds, uint32_t k0, uint64_t behind, bool on, uint32_t wave,
                                         uint32_t lane, int from = 0, int to = kLoads,
                                         uint32_t left = 64) const {
#ifdef __HIP_DEVICE_COMPILE__  // the host's pass knows no 16-byte loads to LDS
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char *>(base + 2 * (k0 + behind)), 0, on ? int(bytes - 2 * k0) : 0, 0x00020000);
#pragma unroll
        for (int j = 0; j < kLoads; j++)
            if (j >= from && j < to) {
                const uint32_t v = TAIL && column(wave, lane, j) >= left ? kNever : at[j];
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rsrc, (lds_void *)(lds + (wave * kLoads + j) * 1024), 16, v, 0, 0, 0);
            }
#endif
    }
    // the operand of lane l: row l % 16 of fragment f, k 8 (l / 16) .. + 7 of half stage kk
    static __device__ __forceinline__ bf16x8 read(const char *lds, uint32_t row, int f, uint32_t kk,
                                                  uint32_t lane) {
        const uint32_t at = (lane & 15u) * 128 + (((4 * kk + (lane >> 4)) ^ (lane >> 1 & 7u)) << 4);
        return *reinterpret_cast<const bf16x8 *>(lds + row * 128 + f * 2048 + at);
    }
};

// A tile's operand whose rows are k: 64 rows of ROWS columns, which a
// transposing read turns: of 16 lanes each names 4 columns of one of 4 rows,
// and receives one column of the 4.  Two neighbouring chunks of 16 bytes stay
// together, and pair p of row k lies in pair slot p ^ turn(k), so that the
// reads of 8 rows (half a wave) fall into different banks.
template <int ROWS, int WAVES>
struct Turned {
    static constexpr int kLoads = ROWS / 8 / WAVES;
    static constexpr uint32_t kChunks = ROWS / 8;  // of a row
    const char *base;
    uint64_t step;  // bytes of a row
    uint32_t gap, at[kLoads];  // gap: what lies between the last row's end and a next one
    static __device__ __forceinline__ uint32_t turn(uint32_t k) {
        if constexpr (ROWS >= 128) return (k & 3u) | (k >> 3 & 1u) << 2;
        else if constexpr (ROWS == 64) return (k >> 1 & 1u) | (k >> 3 & 1u) << 1;
        else return k >> 3 & 1u;
    }
    // columns from `p` on, `left` of them up to the row's end
    __device__ void init(const __bf16 *p, uint64_t stride, uint32_t left, uint32_t, uint32_t wave,
                         uint32_t lane) {
        base = reinterpret_cast<const char *>(p);
        step = 2 * stride;
        gap = uint32_t(step) - 2 * left;
#pragma unroll
        for (int j = 0; j < kLoads; j++) {
            const uint32_t slot = (wave * kLoads + j) * 64 + lane, k = slot / kChunks;
            const uint32_t chunk = slot % kChunks ^ turn(k) << 1;
            at[j] = k * uint32_t(step) + chunk * 16;
        }
    }
    // rows k0 .. k0 + 63 of `rows` to LDS, zeros past the end
    __device__ __forceinline__ void load(char *lds, uint32_t k0, uint32_t rows, uint64_t half,
                                         uint32_t wave, int from = 0, int to = kLoads) const {
#ifdef __HIP_DEVICE_COMPILE__
        const uint32_t here = k0 < rows ? min(rows - k0, kDepth) : 0;
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char *>(base + k0 * step + 2 * half), 0,
            here ? int(here * uint32_t(step) - gap) : 0, 0x00020000);
#pragma unroll
        for (int j = 0; j < kLoads; j++)
            if (j >= from && j < to)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rsrc, (lds_void *)(lds + (wave * kLoads + j) * 1024), 16, at[j], 0, 0, 0);
#endif
    }
    static __device__ __forceinline__ bf16x8 read(const char *lds, uint32_t row, int f, uint32_t kk,
                                                  uint32_t lane) {
        union {
            s16x4 half[2];
            bf16x8 all;
        } v;
#ifdef __HIP_DEVICE_COMPILE__
        const uint32_t k = 8 * (lane >> 4) + ((lane & 15u) >> 2);
        const char *p = lds + (32 * kk + k) * (2 * ROWS) + ((row / 16 + f) ^ turn(k)) * 32 + (lane & 3u) * 8;
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        v.half[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
        v.half[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * 2 * ROWS));
#endif
        return v.all;
    }
};

// The hardware's power of 2, which is good to 1 in 2^23, of a product rounded to float32:
// the argument's rounding moves the exponential by up to |x| 2^-23 of itself (x = -20: 2.4e-6
// of 2e-9), less than the logits' own roundings do, which lse and g have in any case.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// Two parts' largest value and sum of exponentials of what lies below it.
__device__ __forceinline__ float2 joined(float2 r, float2 o) {
    const float top = fmaxf(r.x, o.x), from = top == -__builtin_inff() ? 0.0f : top;
    return make_float2(top, r.y * exp_of(r.x - from) + o.y * exp_of(o.x - from));
}

// Y: what is stored; S: what the results are until then.
template <class Y, class S, int KIND, int BT, int BR, int WT, int WR, int NB>
__global__ __launch_bounds__(64 * WT * WR) void tiles(TileArgs a) {
    constexpr int kWaves = WT * WR, FT = BT / WT / 16, FR = BR / WR / 16;
    constexpr bool kLogits = KIND == STATS || KIND == GRAD, kDw = KIND >= DW;
    using A = std::conditional_t<kDw, Turned<BT, kWaves>, Straight<BT, kWaves>>;
    using B = std::conditional_t<kLogits, Straight<BR, kWaves>, Turned<BR, kWaves>>;
    constexpr int kA = BT * kDepth * 2, kB = BR * kDepth * 2;  // bytes of a stage
    // a buffer is an object of its own, so that the compiler sees that reads
    // of one do not wait for loads to another
    __shared__ __align__(16) char x0[kA], w0[kB], x1[kA], w1[kB];
    __shared__ __align__(16) char x2[NB > 2 ? kA : 16], w2[NB > 2 ? kB : 16];
    __shared__ __align__(16) char x3[NB > 3 ? kA : 16], w3[NB > 3 ? kB : 16];
    __shared__ __align__(16) char x4[NB > 4 ? kA : 16], w4[NB > 4 ? kB : 16];
    __shared__ __align__(16) char x5[NB > 4 ? kA : 16], w5[NB > 4 ? kB : 16];
    static_assert(held(BT, BR) && held(BT, BR) * (NB * (kA + kB) + BT * 16 + 128) <= 160 * 1024,
                  "a compute unit's LDS holds the workgroups that the tile's times are for");
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = uniform(threadIdx.x >> 6);
    // tokens that there are, where only the device knows
    const uint32_t n = a.count ? uniform(*a.count) : 0;
    const uint32_t t_size = !kDw && a.count ? n : a.t_size;
    const uint32_t k_size = kDw ? n : a.k_size;

    // Workgroups go to the 8 XCDs in turn: every XCD takes one run of the
    // tiles and walks them 4 wide in t, so that the tiles at work on an XCD
    // share both operands in its L2
    const uint32_t t_tiles = (t_size + BT - 1) / BT, r_tiles = (a.r_size + BR - 1) / BR;
    const uint32_t all = t_tiles * r_tiles * a.splits, run = (all + 7) / 8;
    const uint32_t turn = blockIdx.x / 8, in_all = blockIdx.x % 8 * run + turn;
    if (turn >= run || in_all >= all) return;
    const uint32_t split = uniform(in_all / (t_tiles * r_tiles)), in = in_all % (t_tiles * r_tiles);
    const uint32_t band = 4 * r_tiles, t_first = in / band * 4, width = min(4u, t_tiles - t_first);
    const uint32_t r_tile = uniform((in % band) / width);
    const uint32_t r0 = r_tile * BR;
    const uint32_t t0 = uniform((t_first + (in % band) % width) * BT);

    A xa;
    B wb;
    if constexpr (kDw) xa.init(a.a + t0, a.a_stride, uint32_t(a.a_stride) - t0, 0, wave, lane);
    else
        xa.init(a.a + t0 * a.a_stride, a.a_stride, t_size - t0, KIND == DX ? uint32_t(a.a_stride) : k_size, wave,
                lane);
    if constexpr (kLogits) wb.init(a.b + r0 * a.b_stride, a.b_stride, a.r_size - r0, k_size, wave, lane);
    else wb.init(a.b + r0, a.b_stride, a.r_size - r0, 0, wave, lane);
    const uint32_t wt = wave / WR * (BT / WT), wr = wave % WR * (BR / WR);
    f32x4 acc[FT][FR];
#pragma unroll
    for (int f = 0; f < FT; f++)
#pragma unroll
        for (int h = 0; h < FR; h++) acc[f][h] = 0.0f;

    // Logits: stage 0 is the last 8 .. 64 columns, stage s > 0 starts at column
    // 64 (s - 1).  The others' stages go over whole groups of 64 (loads give zeros
    // behind the end of k), a split's own, each once for every term of g, so that
    // the other operand comes from the cache after the first (16 tokens, 128256 x
    // 4096, two terms: 1029 us where the second term followed the first, 911 so).
    const uint32_t whole = (k_size + kDepth - 1) / kDepth;
    const uint32_t s_first = kLogits ? 0 : min(whole, split * a.split_stages);
    const uint32_t s_here = kLogits ? whole : min(whole - s_first, a.split_stages);
    const uint32_t stages = kLogits ? s_here : s_here * a.terms;
    // where the next stage to be loaded lies, of those of DX and DW, and the term of g
    uint32_t next_k = s_first * kDepth, next_term = 0;
    const uint32_t end_k = next_k + s_here * kDepth;
    const auto load_a = [&](char *lds, uint32_t s, int from, int to) {
        if constexpr (kLogits) {
            xa.load(lds, (s - 1) * kDepth, 0, s < stages, wave, lane, from, to);
        } else {
            const uint64_t behind = next_term * a.a_term;
            if constexpr (KIND == DX) xa.load(lds, next_k, behind, next_k < end_k, wave, lane, from, to);
            else xa.load(lds, next_k, next_k < end_k ? k_size : 0, behind, wave, from, to);
        }
    };
    const auto load_b = [&](char *lds, uint32_t s, int from, int to) {
        if constexpr (kLogits) wb.load(lds, (s - 1) * kDepth, 0, s < stages, wave, lane, from, to);
        else wb.load(lds, next_k, next_k < end_k ? k_size : 0, 0, wave, from, to);
    };
    const auto load_both = [&](char *xs, char *ws, uint32_t s) {
        load_b(ws, s, 0, B::kLoads);
        load_a(xs, s, 0, A::kLoads);
        if (!kLogits && ++next_term == a.terms) next_term = 0, next_k += kDepth;
    };

    // A step of 32 of k multiplies one set of operands while the next set
    // is read from LDS; before a stage's last step its waves meet: the next
    // stage has arrived then, and this one's buffer is free for the one after
    // it, whose loads go out at once (between the products of that step, as they
    // did before, leaves them less time: 8192 x 65536 logits 3161 -> 3070 us).  The
    // scheduling barriers hold the reads between the products.
    struct Operands {
        bf16x8 x[FT], w[FR];
    } even, odd;
    const auto read = [&](Operands &o, const char *xs, const char *ws, uint32_t kk, int f) {
        if (f < FT) o.x[f] = A::read(xs, wt, f, kk, lane);
        if (f < FR) o.w[f] = B::read(ws, wr, f, kk, lane);
    };
    constexpr int kF = FT > FR ? FT : FR;
    const auto products = [&](const Operands &o, int f) {
        __builtin_amdgcn_sched_barrier(0);
        if (f < FT) {
#pragma unroll
            for (int h = 0; h < FR; h++)
                acc[f][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(o.w[h], o.x[f], acc[f][h], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int XL = A::kLoads, WL = B::kLoads;
    // the next stage has arrived when at most the loads of the NB - 2 behind it are out
    constexpr int kOut = (NB - 2) * (XL + WL), kStart = (NB - 1) * (XL + WL);
    static_assert(kStart < 64, "the counter of loads");
    const auto arrived = [&] {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((kOut & 15) | (kOut >> 4 << 14) | 0x0070);  // and lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // Loads for stages past the last give zeros, so that the loop has no
    // conditions and the stages that fill up a round of the buffers add nothing.
    const auto stage = [&](char *xs, char *ws, char *xn, char *wn, uint32_t s) {
#pragma unroll
        for (int f = 0; f < kF; f++) {
            read(odd, xs, ws, 1, f);
            products(even, f);
        }
        arrived();
        load_both(xs, ws, s + NB);
#pragma unroll
        for (int f = 0; f < kF; f++) {
            read(even, xn, wn, 0, f);
            products(odd, f);
        }
    };
    // what the results of a token need: its lse, p, q and target's row (of the
    // piece), read first and put into LDS when they have come
    __shared__ float4 tokens[kLogits ? BT : 1];
    float4 token = make_float4(0.0f, 0.0f, 0.0f, __uint_as_float(kNever));
    if (kLogits && threadIdx.x < BT && t0 + threadIdx.x < t_size) {
        const uint32_t t = t0 + threadIdx.x;
        if constexpr (KIND == STATS) {
            const int64_t target = a.target_bits == 64 ? static_cast<const int64_t *>(a.targets)[t]
                                                       : int64_t(static_cast<const int32_t *>(a.targets)[t]);
            if (target >= a.first && target < int64_t(a.first) + a.r_size)
                token.w = __uint_as_float(uint32_t(target) - a.first);
        } else {
            token.x = a.lse[t], token.y = a.factor[t].x, token.z = a.factor[t].y;
            token.w = __uint_as_float(a.target_of[t] - a.first);
        }
    }
    const auto put_token = [&] {
        if (kLogits && threadIdx.x < BT) tokens[threadIdx.x] = token;
    };
    if (!stages) put_token();
    if (stages) {
        if constexpr (kLogits) {
            const uint32_t tail = (stages - 1) * kDepth;
            xa.template load<true>(x0, tail, 0, true, wave, lane, 0, XL, k_size - tail);
            wb.template load<true>(w0, tail, 0, true, wave, lane, 0, WL, k_size - tail);
        } else {
            load_both(x0, w0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        const auto begin = [&](char *xs, char *ws, uint32_t s) {
            load_both(xs, ws, s);
            __builtin_amdgcn_sched_barrier(0);
        };
        begin(x1, w1, 1);
        if constexpr (NB > 2) begin(x2, w2, 2);
        if constexpr (NB > 3) begin(x3, w3, 3);
        if constexpr (NB > 4) begin(x4, w4, 4), begin(x5, w5, 5);
        put_token();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((kStart & 15) | (kStart >> 4 << 14) | 0x0070);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
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
    // the stages' buffers are free once the last loads, of zeros, have come
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
    __syncthreads();

    // Lane l holds t l % 16 and r 4 (l / 16) .. + 3 of each product.
    const uint32_t q = lane >> 4, i = lane & 15u;
    const bool edge = r0 + BR > a.r_size || t0 + BT > t_size;
    if constexpr (KIND == STATS) {
        float2 *both = reinterpret_cast<float2 *>(x0);  // [wave of r][t]
        static_assert(WR * BT * 8 <= kA, "room for the waves' sums");
#pragma unroll
        for (int f = 0; f < FT; f++) {
            // the target's logit, where it is this wave's, leaves the others
            const uint32_t target = __float_as_uint(tokens[wt + 16 * f + i].w) - r0 - wr;
            if (__any(target < 16 * FR)) {
                float told = 0.0f;
#pragma unroll
                for (int h = 0; h < FR; h++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const bool is = target == 16 * h + 4 * q + e;
                        told = is ? acc[f][h][e] : told;
                        acc[f][h][e] = is ? -__builtin_inff() : acc[f][h][e];
                    }
                if (target < 16 * FR && (target >> 2 & 3) == q) a.told[t0 + wt + 16 * f + i] = told;
            }
            if (edge) {
#pragma unroll
                for (int h = 0; h < FR; h++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (r0 + wr + 16 * h + 4 * q + e >= a.r_size) acc[f][h][e] = -__builtin_inff();
            }
            float top = -__builtin_inff();
#pragma unroll
            for (int h = 0; h < FR; h++)
#pragma unroll
                for (int e = 0; e < 4; e++) top = fmaxf(top, acc[f][h][e]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float from = top == -__builtin_inff() ? 0.0f : top;
            float sum = 0.0f;
#pragma unroll
            for (int h = 0; h < FR; h++)
#pragma unroll
                for (int e = 0; e < 4; e++) sum += exp_of(acc[f][h][e] - from);
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (q == 0) both[wave % WR * BT + wt + 16 * f + i] = make_float2(top, sum);
        }
        __syncthreads();
        for (uint32_t t = threadIdx.x; t < BT; t += 64 * kWaves) {
            if (t0 + t >= t_size) break;
            float2 r = both[t];
#pragma unroll
            for (int p = 1; p < WR; p++) r = joined(r, both[p * BT + t]);
            const uint32_t at = t0 + t;
            a.part[(uint64_t(at / 16) * a.part_tiles + r_tile) * 16 + at % 16] = r;
        }
        return;
    } else {
        // The results pass through LDS, 128 bytes of each of 32 t at a time, so
        // that a t's leave in whole cache lines.
        constexpr int kRows = std::min<int>(128 / sizeof(S), 16 * FR), kParts = kRows / 16;
        constexpr uint32_t kBytes = kRows * sizeof(S), kPitch = kBytes + 16;  // t's in different banks
        // A wave's 32 t in stages' buffers, which are free now: memory of their own
        // would leave a compute unit room for one workgroup of the small tiles, not two
        // (gradient of 16 tokens, 128256 x 4096: dx 296 us, 279 in the buffers)
        constexpr uint32_t kX = kA / (32 * kPitch), kW = kB / (32 * kPitch);
        static_assert(FR % kParts == 0, "whole rows of results");
        static_assert(kWaves <= 2 * kX + 2 * kW, "room for the waves' results");
        const uint32_t of_w = wave - 2 * kX;
        char *out = wave < 2 * kX ? (wave < kX ? x0 : x1) + wave % std::max(kX, 1u) * (32 * kPitch)
                                  : (of_w < kW ? w0 : w1) + of_w % std::max(kW, 1u) * (32 * kPitch);
        constexpr uint32_t kEach = 16 / sizeof(S);
        typedef S S4 __attribute__((ext_vector_type(4)));
        typedef S SE __attribute__((ext_vector_type(kEach)));
        typedef Y YE __attribute__((ext_vector_type(kEach)));
        typedef YE YE_any __attribute__((aligned(sizeof(Y))));
        // what of the tile is stored, where
        const uint32_t r_end = KIND == GRAD ? a.r_padded : a.r_size;
        Y *y = KIND == GRAD ? reinterpret_cast<Y *>(a.g) : static_cast<Y *>(a.y) + split * a.y_split;
        const uint64_t y_stride = KIND == GRAD ? a.g_stride : a.y_stride;
        constexpr uint32_t kLanes = kBytes / 16;  // of a t
        const uint32_t chunk = lane % kLanes;
        const auto store = [&](int f, int h0) {
            // a wave's LDS operations take effect in order: no barrier
            const uint32_t r = r0 + wr + 16 * h0 + chunk * kEach;
#pragma unroll
            for (uint32_t p = 0; p < kLanes / 2; p++) {
                const uint32_t j = 64 / kLanes * p + lane / kLanes, t = t0 + wt + 32 * f + j;
                const SE v = *reinterpret_cast<const SE *>(out + j * kPitch + chunk * 16);
                if (t >= t_size) continue;
                Y *to = y + t * y_stride + r;
                if (r + kEach <= r_end) {
                    YE sum;
#pragma unroll
                    for (uint32_t e = 0; e < kEach; e++) sum[e] = Y(v[e]);
                    if (KIND == DW_PAST) __builtin_nontemporal_store(YE_any(sum), reinterpret_cast<YE_any *>(to));
                    else *reinterpret_cast<YE_any *>(to) = sum;
                } else {
#pragma unroll
                    for (uint32_t e = 0; e < kEach - 1; e++)
                        if (r + e < r_end) to[e] = Y(v[e]);
                }
            }
        };
        // The same, added to what is there, which is read a store ahead (1001 tokens,
        // 32003 x 1000, dw in float32 of two terms: 424 us without, 409 with that).
        struct Old {
            YE v[kLanes / 2];
        };
        const auto each = [&](int f, int h0, auto use) {
            const uint32_t r = r0 + wr + 16 * h0 + chunk * kEach;
#pragma unroll
            for (uint32_t p = 0; p < kLanes / 2; p++) {
                const uint32_t j = 64 / kLanes * p + lane / kLanes, t = t0 + wt + 32 * f + j;
                use(p, j, y + t * y_stride + r, t >= t_size || r >= r_end ? 0 : min(r_end - r, kEach));
            }
        };
        const auto fetch = [&](int f, int h0) {
            Old old;
            each(f, h0, [&](uint32_t p, uint32_t, const Y *from, uint32_t here) {
                if (here == kEach) {
                    old.v[p] = *reinterpret_cast<const YE_any *>(from);
                } else {
#pragma unroll
                    for (uint32_t e = 0; e < kEach; e++) old.v[p][e] = e < here ? from[e] : Y(0.0f);
                }
            });
            return old;
        };
        const auto store_added = [&](int f, int h0, const Old &old) {
            each(f, h0, [&](uint32_t p, uint32_t j, Y *to, uint32_t here) {
                const SE v = *reinterpret_cast<const SE *>(out + j * kPitch + chunk * 16);
                YE sum;
#pragma unroll
                for (uint32_t e = 0; e < kEach; e++) sum[e] = Y(float(v[e]) + float(old.v[p][e]));
                if (here == kEach) {
                    if (KIND == DW_PAST) __builtin_nontemporal_store(YE_any(sum), reinterpret_cast<YE_any *>(to));
                    else *reinterpret_cast<YE_any *>(to) = sum;
                } else {
#pragma unroll
                    for (uint32_t e = 0; e < kEach - 1; e++)
                        if (e < here) to[e] = sum[e];
                }
            });
        };
        const bool add = KIND != GRAD && a.add;
        const float scale = kDw ? *a.scale : 1.0f;
        Old old{};
        if (add) old = fetch(0, 0);
#pragma unroll
        for (int f = 0; f < FT / 2; f++) {
#pragma unroll
            for (int h0 = 0; h0 < FR; h0 += kParts) {
                if constexpr (KIND == GRAD) {
                    // The part of g, rounded to BF16, which the matrix cores multiply; a
                    // further term is what those before it leave.  One term's error is
                    // below that of the gradient's own rounding to BF16 (drawn shapes, of
                    // the norm: dx 0.00166 -> 0.0020 in the median, 0.0023 at most); a
                    // second costs its products again
#pragma unroll
                    for (int g = 0; g < 2; g++) {
                        const float4 of = tokens[wt + 32 * f + 16 * g + i];
                        const uint32_t target = __float_as_uint(of.w) - r0 - wr;
                        const bool on = t0 + wt + 32 * f + 16 * g + i < t_size;
                        f32x4 (&row)[FR] = acc[2 * f + g];
#pragma unroll
                        for (int h = h0; h < h0 + kParts; h++)
#pragma unroll
                            for (int e = 0; e < 4; e++) row[h][e] = of.y * exp_of(row[h][e] - of.x);
                        if (__any(target < 16 * FR)) {
#pragma unroll
                            for (int h = h0; h < h0 + kParts; h++)
#pragma unroll
                                for (int e = 0; e < 4; e++)
                                    if (target == 16 * h + 4 * q + e)
                                        row[h][e] = a.exact_target ? of.z : row[h][e] - of.z;
                        }
                        if (edge) {
#pragma unroll
                            for (int h = h0; h < h0 + kParts; h++)
#pragma unroll
                                for (int e = 0; e < 4; e++)
                                    if (!on || r0 + wr + 16 * h + 4 * q + e >= a.r_size) row[h][e] = 0.0f;
                        }
                    }
                }
                for (uint32_t term = 0; term < (KIND == GRAD ? a.terms : 1); term++) {
#pragma unroll
                    for (int h = h0; h < h0 + kParts; h++) {
#pragma unroll
                        for (int g = 0; g < 2; g++) {
                            S4 v;
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                v[e] = S(kDw ? acc[2 * f + g][h][e] * scale : acc[2 * f + g][h][e]);
                                if constexpr (KIND == GRAD) acc[2 * f + g][h][e] -= float(v[e]);
                            }
                            *reinterpret_cast<S4 *>(out + (16 * g + i) * kPitch +
                                                    (16 * (h - h0) + 4 * q) * sizeof(S)) = v;
                        }
                    }
                    if (add) {
                        Old next{};
                        if (h0 + kParts < FR) next = fetch(f, h0 + kParts);
                        else if (f + 1 < FT / 2) next = fetch(f + 1, 0);
                        store_added(f, h0, old);
                        old = next;
                    } else {
                        y += term * a.g_term;
                        store(f, h0);
                        y -= term * a.g_term;
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------- tokens

struct TokenArgs {
    const void *targets;
    uint32_t target_bits, n, vocab;
    int64_t ignored;
    // loss_join
    const float2 *part;
    uint32_t part_tiles;
    const float *told;
    float2 *state;
    float *losses, *lse;
    uint32_t begin, end;
    // pick, gather, spread
    const float *lse_in, *loss_in, *loss_grad, *lse_grad;
    uint32_t loss_grad_step, lse_grad_step;
    float loss_grad_all;
    uint32_t *count, *order, *place, *target_of;
    float *scale, *lse_of;
    float2 *factor;
    const __bf16 *x;
    uint64_t x_stride, to_stride;
    __bf16 *to;
    uint32_t cols;
    // spread
    const float *sums;
    uint64_t sums_split;
    uint32_t splits;
    void *dx;
    uint64_t dx_stride;
};

__device__ __forceinline__ int64_t target_at(const TokenArgs &a, uint32_t t) {
    return a.target_bits == 64 ? static_cast<const int64_t *>(a.targets)[t]
                               : int64_t(static_cast<const int32_t *>(a.targets)[t]);
}

// Joins what the tiles of a piece left for 16 tokens, and earlier pieces.  10 us
// for the 2004 tiles of 16 tokens x 128256 rows.
__global__ __launch_bounds__(1024) void loss_join(TokenArgs a) {
    __shared__ float2 both[64][16];
    const uint32_t i = threadIdx.x & 15u, lane = threadIdx.x >> 4, t = blockIdx.x * 16 + i;
    const float2 *part = a.part + uint64_t(blockIdx.x) * a.part_tiles * 16 + i;
    float2 r = make_float2(-__builtin_inff(), 0.0f);
    constexpr uint32_t kLoads = 8;
    for (uint32_t k = lane; t < a.n && k < a.part_tiles; k += 64 * kLoads) {
        float2 v[kLoads];
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++) v[u] = part[min(k + 64 * u, a.part_tiles - 1) * 16];
#pragma unroll
        for (uint32_t u = 0; u < kLoads; u++)
            if (k + 64 * u < a.part_tiles) r = joined(r, v[u]);
    }
    both[lane][i] = r;
    __syncthreads();
#pragma unroll
    for (uint32_t d = 32; d; d >>= 1) {
        if (lane < d) both[lane][i] = r = joined(r, both[lane + d][i]);
        __syncthreads();
    }
    if (lane || t >= a.n) return;
    if (!a.begin) r = joined(a.state[t], r);
    a.state[t] = r;
    if (!a.end) return;
    // o: the logarithm of the others' sum; with d = o - l[target] the loss is
    // log(1 + exp d), which keeps its digits where the target is nearly certain
    const float inf = __builtin_inff(), nan = __builtin_nanf("");
    const float of_sum = r.x == -inf ? 0.0f * r.y : logf(r.y);
    const float o = r.x + of_sum;
    const int64_t target = target_at(a, t);
    if (target < 0 || target >= a.vocab) {
        a.lse[t] = o;
        a.losses[t] = target == a.ignored ? 0.0f : nan;
        return;
    }
    const float told = a.told[t], d = r.x - told + of_sum;
    const float more = log1pf(expf(-fabsf(d)));
    float loss = fmaxf(d, 0.0f) + more, lse = d > 0.0f ? o + more : told + loss;
    if (d != d || told == inf) {  // NaN, an infinite logit, or none above -infinity
        loss = nan;
        lse = o == -inf && told == -inf ? -inf : nan;
    }
    a.lse[t] = lse;
    a.losses[t] = target == a.ignored ? 0.0f : loss;
}

// The gradient of token t's loss.
__device__ __forceinline__ float loss_grad_of(const TokenArgs &a, uint32_t t) {
    return a.loss_grad ? a.loss_grad[t * uint64_t(a.loss_grad_step)] : a.loss_grad_all;
}

// What g is divided by, and dx and dw are multiplied with: 1 to 2, the digits of the
// first counted token's gradient, usually those of all.  The target's entry of a token
// that is not known is then next to a power of two, which BF16 holds, where one of
// 1 / 120 loses 1 in 290, in every token alike and so in dx and dw (drawn shapes, error
// of the norm in BF16: dx 0.0023 in the median and 0.0036 at most, 0.0020 and 0.0023 so;
// dw 0.0021 and 0.0034, 0.0019 and 0.0022 so).
__device__ __forceinline__ float digits(float x) {
    const uint32_t bits = __float_as_uint(x), power = bits >> 23 & 0xFFu;
    return power == 0 || power == 0xFF ? 1.0f : __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u);
}

// What a token's part of g needs, at its place among those that have a gradient.
__device__ __forceinline__ void put_token(const TokenArgs &a, uint32_t t, uint32_t at, int64_t target, float scale) {
    const bool inside = target >= 0 && target < a.vocab;
    const float of_loss = loss_grad_of(a, t) / scale;
    const float of_lse = a.lse_grad ? a.lse_grad[t * uint64_t(a.lse_grad_step)] / scale : 0.0f;
    const float nan = __builtin_nanf("");
    // at the target p (l - lse) - q = of_loss (exp(-loss) - 1) + of_lse exp(-loss)
    float q = of_loss;
    if (a.loss_in) q = of_loss * expm1f(-a.loss_in[t]) + (of_lse == 0.0f ? 0.0f : of_lse * expf(-a.loss_in[t]));
    a.order[at] = t;
    a.target_of[at] = inside ? uint32_t(target) : 0xFFFFFFFFu;
    a.lse_of[at] = a.lse_in[t];
    a.factor[at] = inside ? make_float2(of_loss + of_lse, q) : make_float2(nan, nan);
}

// The tokens that have a gradient, in order.
__global__ __launch_bounds__(1024) void pick(TokenArgs a) {
    __shared__ uint32_t sums[16], firsts[16];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    uint32_t before = 0;
    float scale = 1.0f;
    for (uint32_t t0 = 0; t0 < a.n; t0 += 1024) {
        const uint32_t t = t0 + threadIdx.x;
        const int64_t target = t < a.n ? target_at(a, t) : a.ignored;
        const bool on = t < a.n && target != a.ignored;
        const uint64_t mask = __ballot(on);
        if (lane == 0) sums[wave] = __popcll(mask), firsts[wave] = mask ? t + __builtin_ctzll(mask) : 0;
        __syncthreads();
        uint32_t at = before + __popcll(mask & ((1ull << lane) - 1)), total = 0, first = 0;
        for (uint32_t w = 0; w < 16; w++) {
            if (w < wave) at += sums[w];
            if (total == 0) first = firsts[w];
            total += sums[w];
        }
        if (before == 0 && total) scale = digits(loss_grad_of(a, first));
        before += total;
        __syncthreads();
        if (t < a.n) a.place[t] = on ? at : 0xFFFFFFFFu;
        if (on) put_token(a, t, at, target, scale);
    }
    if (threadIdx.x == 0) *a.count = before, *a.scale = scale;
}

// Their hidden states, one behind the other: a wave for each 512 columns.
__global__ __launch_bounds__(256) void gather(TokenArgs a) {
    const uint32_t parts = (a.cols + 511) / 512;
    const uint32_t wave = uniform(blockIdx.x * 4 + (threadIdx.x >> 6)), lane = threadIdx.x & 63u;
    const uint32_t i = wave / parts, c = wave % parts * 512 + lane * 8;
    if (i >= *a.count || c >= a.cols) return;
    *reinterpret_cast<bf16x8 *>(a.to + i * a.to_stride + c) =
        *reinterpret_cast<const bf16x8 *>(a.x + a.order[i] * a.x_stride + c);
}

// Both in one launch for few tokens: every wave counts those before its own.
constexpr uint32_t kFewTokens = 1024;

__global__ __launch_bounds__(256) void pick_and_gather(TokenArgs a) {
    const uint32_t parts = (a.cols + 511) / 512;
    const uint32_t wave = uniform(blockIdx.x * 4 + (threadIdx.x >> 6)), lane = threadIdx.x & 63u;
    const uint32_t t = wave / parts, c = wave % parts * 512 + lane * 8;
    if (t >= a.n) return;
    const int64_t target = target_at(a, t);
    bf16x8 x;
    if (c < a.cols) x = *reinterpret_cast<const bf16x8 *>(a.x + t * a.x_stride + c);
    uint32_t at = 0, first = t;
    for (uint32_t i0 = 0; i0 < t; i0 += 4 * 64) {
        int64_t other[4];
#pragma unroll
        for (uint32_t u = 0; u < 4; u++) other[u] = target_at(a, min(i0 + 64 * u + lane, t));
#pragma unroll
        for (uint32_t u = 0; u < 4; u++) {
            const uint64_t mask = __ballot(i0 + 64 * u + lane < t && other[u] != a.ignored);
            if (at == 0 && mask) first = i0 + 64 * u + __builtin_ctzll(mask);
            at += __popcll(mask);
        }
    }
    const bool on = target != a.ignored;
    if (on && c < a.cols) *reinterpret_cast<bf16x8 *>(a.to + at * a.to_stride + c) = x;
    if (wave % parts || lane) return;
    a.place[t] = on ? at : 0xFFFFFFFFu;
    const float scale = at + on ? digits(loss_grad_of(a, first)) : 1.0f;
    if (on) put_token(a, t, at, target, scale);
    if (t == a.n - 1) *a.count = at + on, *a.scale = scale;
}

// dx of every token: the splits' sums in order, zeros for those without a gradient.
template <class Y>
__global__ __launch_bounds__(256) void spread(TokenArgs a) {
    const uint32_t parts = (a.cols + 511) / 512;
    const uint32_t wave = uniform(blockIdx.x * 4 + (threadIdx.x >> 6)), lane = threadIdx.x & 63u;
    const uint32_t t = wave / parts, c = wave % parts * 512 + lane * 8;
    if (t >= a.n || c >= a.cols) return;
    const uint32_t at = a.place[t];
    const float scale = *a.scale;
    f32x8 sum = 0.0f;
    if (at != 0xFFFFFFFFu) {
        const float *from = a.sums + at * uint64_t(a.cols) + c;
        constexpr uint32_t kLoads = 8;
        for (uint32_t k = 0; k < a.splits; k += kLoads) {
            f32x8 v[kLoads];
#pragma unroll
            for (uint32_t u = 0; u < kLoads; u++)
                if (k + u < a.splits) v[u] = *reinterpret_cast<const f32x8 *>(from + (k + u) * a.sums_split);
#pragma unroll
            for (uint32_t u = 0; u < kLoads; u++)
                if (k + u < a.splits) sum += v[u];
        }
    }
    store_group<Y>(static_cast<Y *>(a.dx) + t * a.dx_stride, c, a.cols, sum * scale);
}

// ---------------------------------------------------------------- host

uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

constexpr int kTileKinds = sizeof(kTiles) / sizeof(kTiles[0]);
constexpr uint32_t kUnits = 256;  // compute units

uint64_t tiles_of(const Tile &tile, uint64_t t, uint64_t r) {
    return (t + tile.t - 1) / tile.t * ((r + tile.r - 1) / tile.r);
}

// How long a product of t x r results takes, its sums of `stages` stages: rounds
// of the workgroups that the chip holds at once, 3 us for a tile's start and end.
float time_of(const Tile &tile, uint64_t t, uint64_t r, uint64_t stages) {
    const uint64_t tiles = tiles_of(tile, t, r), round = kUnits * tile.held;
    const float rounds = float((tiles + round - 1) / round);
    return tiles <= kUnits ? float(stages) * tile.alone + 3.0f : rounds * (float(stages) * tile.full + 3.0f);
}

// The tile with the least time for a product of t x r results, sums of k.  What it
// decides (logits of 128256 rows, us, tiles of 64 x 128 / 128 x 128 / 256 x 256):
// 64 tokens 193 / 200 / -, 128 tokens - / 233 / 280, 256 tokens - / 354 / 266, 512
// tokens 793 / 666 / 504.
int tile_for(uint64_t t, uint64_t r, uint64_t k) {
    const uint64_t stages = (k + kDepth - 1) / kDepth;
    int best = 0;
    for (int i = 1; i < kTileKinds; i++)
        if (time_of(kTiles[i], t, r, stages) < time_of(kTiles[best], t, r, stages)) best = i;
    return best;
}

// dx's long sums in parts, so that its few tiles fill the chip: the tile, and
// how many parts.  A part writes and reads n x cols floats more (5 TB/s).  512
// tokens x 128256 x 4096: 8 parts of 256 x 256 tiles 483 us, 4 parts of 128 x 128
// 618, one part 1147.
struct Split {
    int tile;
    uint32_t parts;
};
Split dx_split(uint64_t n, uint64_t cols, uint64_t rows) {
    const uint64_t stages = std::max<uint64_t>((rows + kDepth - 1) / kDepth, 1);
    Split best{0, 1};
    float least = 0;
    for (int i = 0; i < kTileKinds; i++) {
        const uint64_t tiles = std::max<uint64_t>(tiles_of(kTiles[i], n, cols), 1);
        const uint64_t most = std::min<uint64_t>({kUnits * kTiles[i].held / tiles, stages / 8, 64});
        const uint64_t parts = std::max<uint64_t>(most, 1);
        const float time = time_of(kTiles[i], n, cols * parts, (stages + parts - 1) / parts) +
                           float(parts * n * cols) * (8 / 5e6f);
        if (i && time >= least) continue;
        least = time;
        best = {i, uint32_t(parts)};
    }
    return best;
}

template <class Y, class S, int KIND>
int run_tiles(int tile, const TileArgs &a, uint64_t t_most, hipStream_t st) {
    const uint64_t all = tiles_of(kTiles[tile], t_most, a.r_size) * a.splits;
    if (!all) return DF11_OK;
    const uint64_t groups = up(all, 8);
    if (groups * kTiles[tile].threads >> 32) return DF11_E_INVALID;  // a grid holds less than 2^32 threads
    const dim3 grid(static_cast<uint32_t>(groups)), block(kTiles[tile].threads);
    switch (tile) {
    case 0: return status(launch(tiles<Y, S, KIND, 32, 64, 1, 2, 6>, grid, block, 0, st, a));
    case 1: return status(launch(tiles<Y, S, KIND, 64, 64, 2, 2, 4>, grid, block, 0, st, a));
    case 2: return status(launch(tiles<Y, S, KIND, 64, 128, 1, 4, 3>, grid, block, 0, st, a));
    case 3: return status(launch(tiles<Y, S, KIND, 128, 128, 4, 2, 4>, grid, block, 0, st, a));
    case 4: return status(launch(tiles<Y, S, KIND, 256, 128, 4, 2, 3>, grid, block, 0, st, a));
    default: return status(launch(tiles<Y, S, KIND, 256, 256, 2, 4, 2>, grid, block, 0, st, a));
    }
}

bool bad_piece(const df11_vocab_piece *p) {
    return !p || p->n > DF11_VOCAB_MAX_TOKENS || p->cols > DF11_VOCAB_MAX_COLS || p->cols % 8 ||
           p->vocab > DF11_VOCAB_MAX_ROWS || p->first > p->vocab || p->rows > p->vocab - p->first ||
           (p->target_bits != 32 && p->target_bits != 64) || p->begin > 1 || p->end > 1 ||
           (p->n && (!p->targets || !aligned(p->targets, p->target_bits / 8))) ||
           p->x_stride % 8 || p->x_stride > DF11_VOCAB_MAX_STRIDE || p->w_stride % 8 ||
           p->w_stride > DF11_VOCAB_MAX_STRIDE ||
           (p->n && p->cols && (!p->x || !aligned(p->x, 16) || (p->n > 1 && p->x_stride < p->cols))) ||
           (p->rows && p->cols && (!p->w || !aligned(p->w, 16) || (p->rows > 1 && p->w_stride < p->cols)));
}

// Places in a caller's scratch, one behind the other.
struct Scratch {
    char *base;
    uint64_t at = 0;
    template <class T>
    T *take(uint64_t n) {
        T *p = reinterpret_cast<T *>(base + at);
        at = up(at + n * sizeof(T), 256);
        return p;
    }
};

// All pieces of a head have the tile of the largest one, whose results have room.
struct LossScratch {
    float2 *state, *part;
    float *told;
    int tile;
    uint64_t bytes;
    LossScratch(void *p, const df11_vocab_sizes &z) : tile(tile_for(z.n, z.rows, z.cols)) {
        Scratch s{static_cast<char *>(p)};
        state = s.take<float2>(z.n);
        told = s.take<float>(z.n);
        part = s.take<float2>(up(z.n, 16) * ((uint64_t(z.rows) + kTiles[tile].r - 1) / kTiles[tile].r));
        bytes = s.at;
    }
};

// g of so many rows at a time: up to 2^29 elements of it (1 GiB, 2 or 3 in two or
// three terms; where the whole of it is less, it takes what logits in as many bytes
// would), in chunks of about the same size.  Every chunk but the first reads and writes dx's sums again: in chunks
// of 2^27 elements 8192 tokens x 128256 x 4096 took 25.32 ms, of 2^29 25.03.
uint64_t chunk_rows(uint64_t n, uint64_t rows) {
    const uint64_t most = std::max<uint64_t>((1ull << 29) / std::max<uint64_t>(n, 1) / 256 * 256, 256);
    const uint64_t chunks = std::max<uint64_t>((rows + most - 1) / most, 1);
    return std::max<uint64_t>(up((rows + chunks - 1) / chunks, 256), 256);
}

// Few tokens have g in two terms also for gradients in BF16: their products wait
// for the head's rows (loss and gradient of 128256 x 4096: 16 tokens 911 us, with
// one term 835; 64 tokens 918 and 848; 128 tokens 1134 and 921), and a sum of few
// products shows a rounding of one of them where they cancel.
constexpr uint32_t kTwoTermTokens = 64;

// Gradients in float32 have it in three, which hold what float32 does: 2e-7 of dw's norm
// and 3e-7 of dx's in the median of drawn shapes, where two terms, 17 bits, left 1.6e-6
// and 2.2e-6 and products in float32 leave 2e-7 and 5e-7.  The third costs its products
// (1001 tokens, 32003 x 1000, dx and dw in float32: 358 -> 472 us).
uint32_t terms_for(uint64_t n, bool f32) { return f32 ? 3 : n <= kTwoTermTokens ? 2 : 1; }

struct GradScratch {
    uint32_t *count, *order, *place, *target_of;
    Split dx;
    float *scale, *lse_of, *sums;
    float2 *factor;
    __bf16 *x, *g;
    uint64_t x_stride, chunk, bytes;
    GradScratch(void *p, const df11_vocab_sizes &z) {
        Scratch s{static_cast<char *>(p)};
        const uint64_t n = z.n;
        count = s.take<uint32_t>(1);
        scale = s.take<float>(1);
        order = s.take<uint32_t>(n), place = s.take<uint32_t>(n), target_of = s.take<uint32_t>(n);
        lse_of = s.take<float>(n);
        factor = s.take<float2>(n);
        x_stride = up(z.cols, 64);
        x = s.take<__bf16>(n * x_stride);
        chunk = chunk_rows(n, z.rows);
        dx = dx_split(n, z.cols, chunk);
        sums = s.take<float>(z.dx ? dx.parts * n * z.cols : 0);
        g = s.take<__bf16>(n * chunk * terms_for(n, z.two_terms));
        bytes = s.at;
    }
};

bool bad_sizes(const df11_vocab_sizes *z) {
    return !z || z->n > DF11_VOCAB_MAX_TOKENS || z->cols > DF11_VOCAB_MAX_COLS || z->cols % 8 ||
           z->rows > DF11_VOCAB_MAX_ROWS;
}

// Whether a piece is not one that the sizes are for.
bool other_sizes(const df11_vocab_piece *p, const df11_vocab_sizes *z) {
    return bad_sizes(z) || z->n != p->n || z->cols != p->cols || p->rows > z->rows;
}

TileArgs tile_args() {
    TileArgs a{};
    a.terms = a.splits = 1;
    a.split_stages = 0xFFFFFFFFu;
    return a;
}

}  // namespace

extern "C" {

uint64_t df11_vocab_loss_scratch_bytes(const df11_vocab_sizes *z) {
    return bad_sizes(z) ? 0 : LossScratch(nullptr, *z).bytes;
}

int df11_vocab_loss(const df11_vocab_piece *p, float *losses, float *lse, const df11_vocab_sizes *sizes,
                    void *scratch, uint64_t scratch_bytes, df11_hip_stream stream) {
    if (bad_piece(p) || !p->vocab || other_sizes(p, sizes)) return DF11_E_INVALID;
    if (!p->n) return DF11_OK;
    const LossScratch s(scratch, *sizes);
    if (!scratch || !aligned(scratch, 256) || scratch_bytes < s.bytes ||
        (p->end && (!losses || !lse || !aligned(losses, 4) || !aligned(lse, 4))))
        return DF11_E_INVALID;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int tile = s.tile;
    TileArgs a = tile_args();
    a.a = static_cast<const __bf16 *>(p->x), a.b = static_cast<const __bf16 *>(p->w);
    a.a_stride = p->x_stride, a.b_stride = p->w_stride;
    a.t_size = p->n, a.r_size = p->rows, a.k_size = p->cols;
    a.targets = p->targets, a.target_bits = p->target_bits, a.first = p->first;
    a.part = s.part, a.told = s.told;
    a.part_tiles = (p->rows + kTiles[tile].r - 1) / kTiles[tile].r;
    int rc = run_tiles<float, float, STATS>(tile, a, p->n, st);
    if (rc != DF11_OK) return rc;
    TokenArgs t{};
    t.targets = p->targets, t.target_bits = p->target_bits, t.n = p->n, t.vocab = p->vocab;
    t.ignored = p->ignored;
    t.part = s.part, t.part_tiles = a.part_tiles, t.told = s.told, t.state = s.state;
    t.losses = losses, t.lse = lse, t.begin = p->begin, t.end = p->end;
    return status(launch(loss_join, dim3((p->n + 15) / 16), dim3(1024), 0, st, t));
}

uint64_t df11_vocab_loss_gradient_scratch_bytes(const df11_vocab_sizes *z) {
    return bad_sizes(z) ? 0 : GradScratch(nullptr, *z).bytes;
}

int df11_vocab_loss_gradient(const df11_vocab_piece *p, const df11_vocab_grad *g,
                             const df11_vocab_sizes *sizes, void *scratch, uint64_t scratch_bytes,
                             df11_hip_stream stream) {
    if (bad_piece(p) || !p->vocab || !g || other_sizes(p, sizes) || g->dx_type > DF11_TYPE_BF16 ||
        g->dw_type > DF11_TYPE_BF16 || g->accumulate > 1)
        return DF11_E_INVALID;
    const bool has_dx = sizes->dx, has_dw = g->dw;
    const uint32_t dx_terms = terms_for(p->n, g->dx_type == DF11_TYPE_F32);
    const uint32_t dw_terms = terms_for(p->n, g->dw_type == DF11_TYPE_F32);
    const uint32_t terms = std::max(has_dx ? dx_terms : 1, has_dw ? dw_terms : 1);
    if (!sizes->two_terms &&
        ((has_dx && g->dx_type == DF11_TYPE_F32) || (has_dw && g->dw_type == DF11_TYPE_F32)))
        return DF11_E_INVALID;
    if (has_dw && (!aligned(g->dw, type_bytes(g->dw_type)) || (p->rows > 1 && g->dw_stride < p->cols) ||
                   g->dw_stride >> 40))
        return DF11_E_INVALID;
    if (p->n && (!g->lse || !aligned(g->lse, 4) || !aligned(g->losses, 4) || !aligned(g->loss_grad, 4) ||
                 !aligned(g->lse_grad, 4) ||
                 (g->loss_grad && g->loss_grads != 1 && g->loss_grads != p->n) ||
                 (g->lse_grad && g->lse_grads != 1 && g->lse_grads != p->n)))
        return DF11_E_INVALID;
    if (has_dx && p->end && p->n && p->cols &&
        (!g->dx || !aligned(g->dx, type_bytes(g->dx_type)) || (p->n > 1 && g->dx_stride < p->cols) ||
         g->dx_stride >> 40))
        return DF11_E_INVALID;
    const GradScratch s(scratch, *sizes);
    if (!scratch || !aligned(scratch, 256) || scratch_bytes < s.bytes) return DF11_E_INVALID;
    if (!p->cols) return DF11_OK;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const uint64_t parts = (p->cols + 511) / 512, waves = p->n * parts;
    if ((waves + 3) >> 26) return DF11_E_INVALID;  // a grid holds less than 2^32 threads
    const dim3 rows(uint32_t((waves + 3) / 4));

    TokenArgs t{};
    t.targets = p->targets, t.target_bits = p->target_bits, t.n = p->n, t.vocab = p->vocab;
    t.ignored = p->ignored;
    t.lse_in = g->lse, t.loss_in = g->losses;
    t.loss_grad = g->loss_grad, t.lse_grad = g->lse_grad, t.loss_grad_all = g->loss_grad_all;
    t.loss_grad_step = g->loss_grads > 1, t.lse_grad_step = g->lse_grads > 1;
    t.count = s.count, t.order = s.order, t.place = s.place, t.target_of = s.target_of;
    t.scale = s.scale, t.lse_of = s.lse_of, t.factor = s.factor;
    t.x = static_cast<const __bf16 *>(p->x), t.x_stride = p->x_stride;
    t.to = s.x, t.to_stride = s.x_stride, t.cols = p->cols;
    int rc = DF11_OK;
    if (p->begin) {
        if (p->n && p->n <= kFewTokens) {
            rc = status(launch(pick_and_gather, rows, dim3(256), 0, st, t));
        } else {
            rc = status(launch(pick, dim3(1), dim3(1024), 0, st, t));
            if (rc == DF11_OK && p->n) rc = status(launch(gather, rows, dim3(256), 0, st, t));
        }
        if (rc != DF11_OK) return rc;
    }
    for (uint64_t c = 0; c < p->rows || (!p->rows && !c); c += s.chunk) {
        const uint32_t here = uint32_t(std::min<uint64_t>(s.chunk, p->rows - c));
        const uint64_t g_stride = up(here, kDepth);
        const __bf16 *w = static_cast<const __bf16 *>(p->w) + c * p->w_stride;
        TileArgs a = tile_args();  // g of these rows
        a.a = s.x, a.a_stride = s.x_stride, a.b = w, a.b_stride = p->w_stride;
        a.count = s.count;
        a.r_size = here, a.k_size = p->cols, a.first = uint32_t(p->first + c);
        a.lse = s.lse_of, a.factor = s.factor, a.target_of = s.target_of;
        a.g = s.g, a.g_stride = g_stride, a.g_term = p->n * g_stride, a.r_padded = uint32_t(g_stride);
        a.terms = terms, a.exact_target = g->losses != nullptr;
        rc = run_tiles<__bf16, __bf16, GRAD>(tile_for(p->n, here, p->cols), a, p->n, st);
        if (rc != DF11_OK) return rc;
        if (has_dx && p->n) {
            a = tile_args();
            a.a = s.g, a.a_stride = g_stride, a.a_term = p->n * g_stride, a.terms = dx_terms;
            a.b = w, a.b_stride = p->w_stride;
            a.count = s.count;
            a.r_size = p->cols, a.k_size = here;
            a.splits = s.dx.parts;
            a.split_stages = uint32_t((g_stride / kDepth + s.dx.parts - 1) / s.dx.parts);
            a.y = s.sums, a.y_stride = p->cols, a.y_split = uint64_t(p->n) * p->cols;
            a.add = !(p->begin && c == 0);
            rc = run_tiles<float, float, DX>(s.dx.tile, a, p->n, st);
            if (rc != DF11_OK) return rc;
        }
        if (has_dw && here) {
            a = tile_args();
            a.a = s.g, a.a_stride = g_stride, a.a_term = p->n * g_stride, a.terms = dw_terms;
            a.b = s.x, a.b_stride = s.x_stride;
            a.count = s.count, a.scale = s.scale;
            a.t_size = here, a.r_size = p->cols;
            a.y_stride = g->dw_stride, a.add = g->accumulate;
            const int tile = tile_for(here, p->cols, uint64_t(p->n) * dw_terms);
            // a gradient that the caches do not hold passes them by, which leaves x and g
            // there (512 tokens, 128256 x 4096: 580 us, 629 through them); float32 only
            // where its rows lie on half lines, as a store's 128 bytes otherwise end in two
            // parts of lines that the caches have to bring together (whole gradient of 64
            // tokens, 56639 rows, dw alone: 4352 columns 302 us past them, 390 through
            // them; 4368 columns 362 and 414; 4360 columns 647 and 447.  In BF16: 512
            // tokens, 128256 x 4104, 1158 and 1226)
            const bool whole = g->dw_type == DF11_TYPE_BF16 || (aligned(g->dw, 64) && g->dw_stride % 16 == 0);
            const bool past = whole && uint64_t(p->rows) * p->cols * type_bytes(g->dw_type) >= 1ull << 27;
            if (g->dw_type == DF11_TYPE_F32) {
                a.y = static_cast<float *>(g->dw) + c * g->dw_stride;
                rc = past ? run_tiles<float, float, DW_PAST>(tile, a, here, st)
                          : run_tiles<float, float, DW>(tile, a, here, st);
            } else {
                a.y = static_cast<__bf16 *>(g->dw) + c * g->dw_stride;
                if (g->accumulate) rc = run_tiles<__bf16, float, DW>(tile, a, here, st);
                else rc = past ? run_tiles<__bf16, __bf16, DW_PAST>(tile, a, here, st)
                               : run_tiles<__bf16, __bf16, DW>(tile, a, here, st);
            }
            if (rc != DF11_OK) return rc;
        }
    }
    if (!has_dx || !p->end || !p->n) return DF11_OK;
    t.sums = s.sums, t.sums_split = uint64_t(p->n) * p->cols, t.splits = s.dx.parts;
    t.dx = g->dx, t.dx_stride = g->dx_stride;
    return status(g->dx_type == DF11_TYPE_F32 ? launch(spread<float>, rows, dim3(256), 0, st, t)
                                              : launch(spread<__bf16>, rows, dim3(256), 0, st, t));
}

}  // extern "C"
