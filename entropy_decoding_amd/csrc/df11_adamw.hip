// AdamW over many tensors, the gradients' norm, and the reader of 8-bit states.
//
// A step is one pass over the tensors: every element's gradient, weight and
// states are read once and written once.  A workgroup takes a chunk of one
// tensor; the table that says which one travels in the kernel arguments, so a
// call needs no device memory of its own.  A lane has 4 elements side by side
// (with 8-bit states two such groups), so that every access of a wave, or of
// its half, is contiguous, and a block of 8-bit states is half a wave, whose
// largest values are five DPP steps away.
//
// What bounds it (8B block, 218 M elements): HBM with 32-bit states, 5.4 - 5.5
// TB/s where a copy of 1 GiB moves 5.1 (BF16 with masters 1120 us, BF16 alone
// 874 us, float32 1123 us); with 8-bit states and masters HBM too (638 us,
// 5.5 TB/s), without masters the vector units (424 - 472 us from run to run, 5.2 -
// 4.6 TB/s; 75 instructions an element).  The norm reads at 6.1 TB/s (71 us), the reader of
// states takes 244 us (5.4 TB/s).  Tensors at odd offsets cost 3 - 7%.
// Streams that pass the caches by gained 4%; one block at a time in a whole
// wave, sqrtf and integer conversions for the codes took 663 us without masters.
//
// Contraction is off: each product and sum is rounded on its own, so that a
// weight does not depend on how the compiler pairs them and an elementwise
// implementation in float32 gives the same bits.
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "df11.h"
#include "df11_launch.h"

#pragma clang fp contract(off)

namespace {

using df11_detail::launch;

constexpr uint32_t kThreads = 256;
constexpr uint32_t kStep = kThreads * 4;    // chunks are multiples of it
constexpr uint32_t kMaxTensors = 36;        // a table of 36 stays below 4 KiB of kernel arguments
constexpr uint32_t kCopies = 16;            // copies of a workgroup's histogram
constexpr uint64_t kMaxNumel = uint64_t(1) << 40;

struct Tensor {
    void *w;
    float *master;
    const void *g;
    void *m, *v;
    float *m_scale, *v_scale;
    unsigned long long *counts;
    uint64_t n;
    float keep, size;  // 1 - lr weight_decay and lr / (1 - b1^t) of a step with host numbers
    double lr_scale, weight_decay;
};

struct Table {
    Tensor t[kMaxTensors];
    uint32_t first[kMaxTensors];  // a tensor's first chunk; 0xFFFFFFFF past the last tensor
    uint32_t chunk;               // elements per chunk, a multiple of kStep
};

struct Numbers {
    float b1, c1, b2, c2, eps;  // c = 1 - b
    float inv_root;             // 1 / sqrt(1 - b2^t)
    double lr, log_b1, log_b2, bias1;
    const float *d_lr;
    const uint64_t *d_step;
    const float *d_factor;
    uint64_t step;
    // of a call that counts the steps made: the number of steps skipped, and what
    // a step that changes nothing adds to which counter (last launch of the call)
    const uint64_t *d_skipped;
    unsigned long long *d_count;
    unsigned long long more;
};

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32_any __attribute__((aligned(1)));

// A lane's 4 elements of the 256 at p: all of them, or those below `left`
// (zeros behind).  The hardware takes any alignment.  Everything is touched
// once a step, so loads and stores pass the caches by.
template <bool WHOLE>
__device__ __forceinline__ f32x4 load4(const float *p, uint32_t i, uint32_t left) {
    if (WHOLE) return __builtin_nontemporal_load(reinterpret_cast<const f32x4_any *>(p + i));
    f32x4 x = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t k = 0; k < 4; k++)
        if (i + k < left) x[k] = p[i + k];
    return x;
}
template <bool WHOLE>
__device__ __forceinline__ f32x4 load4(const __bf16 *p, uint32_t i, uint32_t left) {
    if (WHOLE)
        return __builtin_convertvector(
            __builtin_nontemporal_load(reinterpret_cast<const bf16x4_any *>(p + i)), f32x4);
    f32x4 x = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t k = 0; k < 4; k++)
        if (i + k < left) x[k] = float(p[i + k]);
    return x;
}
template <bool WHOLE>
__device__ __forceinline__ uint32_t load4(const uint8_t *p, uint32_t i, uint32_t left) {
    if (WHOLE) return __builtin_nontemporal_load(reinterpret_cast<const u32_any *>(p + i));
    uint32_t x = 0;
#pragma unroll
    for (uint32_t k = 0; k < 4; k++)
        if (i + k < left) x |= uint32_t(p[i + k]) << (8 * k);
    return x;
}
template <bool WHOLE>
__device__ __forceinline__ void store4(float *p, uint32_t i, uint32_t left, f32x4 x) {
    if (WHOLE) {
        __builtin_nontemporal_store(f32x4_any(x), reinterpret_cast<f32x4_any *>(p + i));
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < 4; k++)
        if (i + k < left) p[i + k] = x[k];
}
template <bool WHOLE>
__device__ __forceinline__ void store4(__bf16 *p, uint32_t i, uint32_t left, bf16x4 x) {
    if (WHOLE) {
        __builtin_nontemporal_store(bf16x4_any(x), reinterpret_cast<bf16x4_any *>(p + i));
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < 4; k++)
        if (i + k < left) p[i + k] = x[k];
}
template <bool WHOLE>
__device__ __forceinline__ void store4(__bf16 *p, uint32_t i, uint32_t left, f32x4 x) {
    store4<WHOLE>(p, i, left, __builtin_convertvector(x, bf16x4));
}
template <bool WHOLE>
__device__ __forceinline__ void store4(uint8_t *p, uint32_t i, uint32_t left, uint32_t x) {
    if (WHOLE) {
        __builtin_nontemporal_store(x, reinterpret_cast<u32_any *>(p + i));
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < 4; k++)
        if (i + k < left) p[i + k] = uint8_t(x >> (8 * k));
}

// The largest x of each half of the wave, in all its lanes (DPP inside rows of
// 16 lanes, then from each half's first row to its second).
__device__ __forceinline__ uint32_t half_max(uint32_t x) {
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x111, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x112, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x114, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x118, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x142, 0xA, 0xF, false)));
    const int lower = __builtin_amdgcn_readlane(int(x), 31), upper = __builtin_amdgcn_readlane(int(x), 63);
    return uint32_t((threadIdx.x & 32u) ? upper : lower);
}

// r = sqrt(x) of N x 4 values, correctly rounded as sqrtf's.  For values in the
// middle of the range two Newton steps from the reciprocal root do that in 11
// instructions, against 20 with sqrtf's scaling and last-place checks; a wave
// with another value (0, NaN) takes sqrtf.  Bits of values that are not
// negative compare as the values do, with NaN above all.
template <int N>
__device__ __forceinline__ void roots(const f32x4 (&x)[N], f32x4 (&r)[N]) {
    uint32_t least = 0xFFFFFFFFu, most = 0;
#pragma unroll
    for (int j = 0; j < N; j++) {
#pragma unroll
        for (int k = 0; k < 4; k++) {
            least = min(least, __float_as_uint(x[j][k]));
            most = max(most, __float_as_uint(x[j][k]));
            const float y = __builtin_amdgcn_rsqf(x[j][k]);
            float s = x[j][k] * y, h = 0.5f * y;
            const float e = __builtin_fmaf(-h, s, 0.5f);
            s = __builtin_fmaf(s, e, s);
            h = __builtin_fmaf(h, e, h);
            r[j][k] = __builtin_fmaf(__builtin_fmaf(-s, s, x[j][k]), h, s);
        }
    }
    if (__builtin_amdgcn_ballot_w64(least < __float_as_uint(0x1p-96f) ||
                                    most > __float_as_uint(0x1p96f))) {
#pragma unroll
        for (int j = 0; j < N; j++) {
#pragma unroll
            for (int k = 0; k < 4; k++) r[j][k] = sqrtf(x[j][k]);
        }
    }
}

// The codes sign(x) round(sqrt(|x| inv)) of 4 values, a byte each, ties to even;
// AT_LEAST_1: 1 instead of 0 where x > 0.  A number below 2^22 added to
// 1.5 2^23 is rounded to an integer, whose two's complement is then the low
// bits.  The hardware's root is off by one in the last place at most, which
// the rounding forgets unless the root lies next to a half; then, and where a
// code of 0 needs the look at x, the wave takes the exact root.  No code passes
// its largest: the largest |x| inv is 127^2 or 255^2 but for three roundings.
template <bool AT_LEAST_1>
__device__ __forceinline__ uint32_t root_codes(f32x4 x, float inv) {
    constexpr float kInt = 0x1.8p23f;
    f32x4 c;
    float far = 0.0f, least = 1.0f;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        float s = __builtin_amdgcn_sqrtf(fabsf(x[k]) * inv);
        if (AT_LEAST_1) least = fminf(least, s);
        else s = __builtin_copysignf(s, x[k]);
        c[k] = s + kInt;
        far = fmaxf(far, fabsf((c[k] - kInt) - s));
    }
    if (__builtin_amdgcn_ballot_w64(far > 0.4999f || (AT_LEAST_1 && least < 0.51f))) {
#pragma unroll
        for (int k = 0; k < 4; k++) {
            float s = rintf(sqrtf(fabsf(x[k]) * inv));
            if (AT_LEAST_1 && x[k] > 0.0f) s = fmaxf(s, 1.0f);
            c[k] = (AT_LEAST_1 ? s : __builtin_copysignf(s, x[k])) + kInt;
        }
    }
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(c[1]), __float_as_uint(c[0]), 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(c[3]), __float_as_uint(c[2]), 0x04000C0Cu);
    return lo | hi;
}

// The scale of a lane's block from the bits of its largest magnitude
// (magnitudes compare as their bits do, and NaN above all), and its reciprocal:
// 0 for a block of zeros, and for one that is not finite, whose scale is NaN.
// unit = 1 / 127^2 or 1 / 255^2, rounded.
struct Scale {
    float s, inv;
    __device__ Scale(uint32_t top, float unit, float tiny) {
        const float x = __uint_as_float(top);
        const bool bad = top >= 0x7F800000u, none = x < tiny;
        s = bad ? __uint_as_float(0x7FC00000u) : none ? 0.0f : x * unit;
        inv = bad || none ? 0.0f : 1.0f / s;
    }
};

// the values of 4 codes (squares of codes are exact)
__device__ __forceinline__ void decode(uint32_t mc, uint32_t vc, float ms, float vs, f32x4 &m, f32x4 &v) {
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const float a = float(int8_t(mc >> (8 * k))), b = float(uint8_t(vc >> (8 * k)));
        m[k] = ms * (a * fabsf(a));
        const float r = vs * (b * b);
        v[k] = r * r;
    }
}

__device__ __forceinline__ const Tensor &find(const Table &a, uint32_t &chunk) {
    uint32_t k = 0;
#pragma unroll
    for (uint32_t j = 1; j < kMaxTensors; j++) k += uint32_t(blockIdx.x >= a.first[j]);
    chunk = blockIdx.x - a.first[k];
    return a.t[k];
}

__device__ __forceinline__ uint64_t counter(const uint64_t *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <class W, bool MASTER, class G, int BITS, bool COUNTS>
__global__ __launch_bounds__(kThreads) void adamw(Table a, Numbers c) {
    __shared__ uint32_t hist[COUNTS ? 256 * (kCopies + 1) : 1];
    uint32_t chunk;
    const Tensor &t = find(a, chunk);
    const uint64_t lo = uint64_t(chunk) * a.chunk;
    const uint64_t n = t.n;
    const uint64_t hi = min(n, lo + a.chunk);
    const bool counting = COUNTS && t.counts;
    if (COUNTS) {
        for (uint32_t s = threadIdx.x; s < 256 * (kCopies + 1); s += kThreads) hist[s] = 0;
        __syncthreads();
    }

    // Steps skipped are rare: the host's factors hold while there are none.  The
    // counters are read by every workgroup and written by one, only in a step
    // that uses neither.
    float keep = t.keep, size = t.size, inv_root = c.inv_root, f = 1.0f;
    const uint64_t skipped = c.d_skipped ? counter(c.d_skipped) : 0;
    if (c.d_lr || c.d_step || skipped) {
        const double lr = (c.d_lr ? double(*c.d_lr) : c.lr) * t.lr_scale;
        double bias1 = c.bias1;
        if (c.d_step || skipped) {
            const double step = double(c.d_step ? counter(c.d_step) : skipped < c.step ? c.step - skipped : 1);
            bias1 = 1.0 - exp(step * c.log_b1);
            inv_root = float(1.0 / sqrt(1.0 - exp(step * c.log_b2)));
        }
        keep = float(1.0 - lr * t.weight_decay);
        size = float(lr / bias1);
    }
    bool still = false;  // the step changes nothing
    if (c.d_factor) {
        f = *c.d_factor;
        still = !(fabsf(f) < __builtin_inff());
        if (still && c.d_count && blockIdx.x == 0 && threadIdx.x == 0) atomicAdd(c.d_count, c.more);
    }

    // A wave's next elements from `at` on, all of them or `left`: NG groups of 4
    // a lane.  With 8-bit states each half of the wave holds a block, so that
    // what a block costs (its reductions, its scales) is shared by 8 elements.
    constexpr int NG = BITS == 8 ? 2 : 1;
    constexpr uint32_t kWave = 256 * NG;
    const uint32_t lane = threadIdx.x & 63u, half = NG == 2 ? lane >> 5 : 0u;
    const uint32_t i0 = NG == 2 ? 256 * half + 4 * (lane & 31u) : 4 * lane;  // + 128 a group
    const uint32_t copy = threadIdx.x % kCopies;
    const auto count = [&](bf16x4 shown, uint32_t i, uint32_t left) {
        const uint16_t *bits = reinterpret_cast<const uint16_t *>(&shown);
#pragma unroll
        for (uint32_t k = 0; k < 4; k++)
            if (i + k < left) atomicAdd(&hist[((bits[k] >> 7) & 0xFFu) * (kCopies + 1) + copy], 1u);
    };
    const auto update = [&](auto whole, uint64_t at, uint32_t left) {
        constexpr bool WHOLE = decltype(whole)::value;
        W *w = static_cast<W *>(t.w) + at;
        float *master = t.master + at;
        f32x4 g[NG], x[NG], m[NG], v[NG], r[NG];
        float *m32 = static_cast<float *>(t.m) + at, *v32 = static_cast<float *>(t.v) + at;
        uint8_t *m8 = static_cast<uint8_t *>(t.m) + at, *v8 = static_cast<uint8_t *>(t.v) + at;
        const uint64_t block = at / DF11_ADAMW_BLOCK + half;
        const bool mine = WHOLE || 256 * half < left;  // the lane's block exists
        uint32_t mc[NG], vc[NG];
#pragma unroll
        for (int j = 0; j < NG; j++) {
            const uint32_t i = i0 + 128 * j;
            g[j] = load4<WHOLE>(static_cast<const G *>(t.g) + at, i, left);
            if constexpr (MASTER) x[j] = load4<WHOLE>(static_cast<const float *>(master), i, left);
            else x[j] = load4<WHOLE>(static_cast<const W *>(w), i, left);
            if constexpr (BITS == 32) {
                m[j] = load4<WHOLE>(static_cast<const float *>(m32), i, left);
                v[j] = load4<WHOLE>(static_cast<const float *>(v32), i, left);
            } else {
                mc[j] = load4<WHOLE>(static_cast<const uint8_t *>(m8), i, left);
                vc[j] = load4<WHOLE>(static_cast<const uint8_t *>(v8), i, left);
            }
        }
        if constexpr (BITS == 8) {
            const float ms = mine ? t.m_scale[block] : 0.0f, vs = mine ? t.v_scale[block] : 0.0f;
#pragma unroll
            for (int j = 0; j < NG; j++) decode(mc[j], vc[j], ms, vs, m[j], v[j]);
        }
#pragma unroll
        for (int j = 0; j < NG; j++) {
            if (c.d_factor) {
#pragma unroll
                for (int k = 0; k < 4; k++) g[j][k] = g[j][k] * f;
            }
#pragma unroll
            for (int k = 0; k < 4; k++) {
                m[j][k] = m[j][k] * c.b1 + g[j][k] * c.c1;
                v[j][k] = v[j][k] * c.b2 + (g[j][k] * c.c2) * g[j][k];
            }
        }
        roots(v, r);
#pragma unroll
        for (int j = 0; j < NG; j++) {
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const float u = m[j][k] / (r[j][k] * inv_root + c.eps);
                x[j][k] = x[j][k] * keep - u * size;
            }
        }
        if constexpr (BITS == 8) {
            uint32_t tm = 0, tr = 0;
#pragma unroll
            for (int j = 0; j < NG; j++) {
#pragma unroll
                for (uint32_t k = 0; k < 4; k++) {
                    if (!WHOLE && i0 + 128 * j + k >= left) m[j][k] = r[j][k] = 0.0f;
                    tm = max(tm, __float_as_uint(m[j][k]) & 0x7FFFFFFFu);
                    tr = max(tr, __float_as_uint(r[j][k]) & 0x7FFFFFFFu);
                }
            }
            const Scale sm(half_max(tm), 1.0f / (127.0f * 127.0f), 0x1p-100f);
            const Scale sv(half_max(tr), 1.0f / (255.0f * 255.0f), 0x1p-149f);
#pragma unroll
            for (int j = 0; j < NG; j++) {
                mc[j] = root_codes<false>(m[j], sm.inv);
                vc[j] = root_codes<true>(r[j], sv.inv);
                mc[j] = sm.inv > 0.0f ? mc[j] : 0u;
                vc[j] = sv.inv > 0.0f ? vc[j] : 0u;
            }
            if ((lane & 31u) == 0 && mine) {
                t.m_scale[block] = sm.s;
                t.v_scale[block] = sv.s;
            }
        }
#pragma unroll
        for (int j = 0; j < NG; j++) {
            const uint32_t i = i0 + 128 * j;
            if constexpr (BITS == 32) {
                store4<WHOLE>(m32, i, left, m[j]);
                store4<WHOLE>(v32, i, left, v[j]);
            } else {
                store4<WHOLE>(m8, i, left, mc[j]);
                store4<WHOLE>(v8, i, left, vc[j]);
            }
            if constexpr (MASTER) store4<WHOLE>(master, i, left, x[j]);
            if constexpr (sizeof(W) == 2) {
                const bf16x4 shown = __builtin_convertvector(x[j], bf16x4);
                store4<WHOLE>(w, i, left, shown);
                if (counting) count(shown, i, left);
            } else {
                store4<WHOLE>(w, i, left, x[j]);
            }
        }
    };
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (!still) {
        for (uint64_t at = lo + kWave * wave; at < hi; at += kWave * (kThreads / 64)) {
            if (at + kWave <= hi) update(std::true_type{}, at, kWave);
            else update(std::false_type{}, at, uint32_t(hi - at));
        }
    } else if (counting) {
        for (uint64_t at = lo + 256 * wave; at < hi; at += kStep) {
            const uint32_t left = uint32_t(min(hi - at, uint64_t(256)));
            count(__builtin_convertvector(load4<false>(static_cast<const W *>(t.w) + at, 4 * lane, left),
                                          bf16x4), 4 * lane, left);
        }
    }
    if (COUNTS) {
        __syncthreads();
        if (counting) {
            uint32_t sum = 0;
            for (uint32_t k = 0; k < kCopies; k++) sum += hist[threadIdx.x * (kCopies + 1) + k];
            if (sum) atomicAdd(&t.counts[threadIdx.x], (unsigned long long)sum);
        }
    }
}

__global__ __launch_bounds__(256) void clear_counts(Table a) {
    unsigned long long *p = a.t[blockIdx.x].counts;
    if (p) p[threadIdx.x] = 0;
}

// m and v of 8-bit states; the outputs travel in the table's w and master.  A
// wave takes 512 elements at a time, 8 a lane, so that BF16 values leave 16
// bytes a lane.
typedef __bf16 bf16x8_any __attribute__((ext_vector_type(8), aligned(2)));
typedef float f32x8_any __attribute__((ext_vector_type(8), aligned(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

__device__ __forceinline__ void store8(float *p, f32x8 x) {
    __builtin_nontemporal_store(f32x8_any(x), reinterpret_cast<f32x8_any *>(p));
}
__device__ __forceinline__ void store8(__bf16 *p, f32x8 x) {
    __builtin_nontemporal_store(__builtin_convertvector(x, bf16x8_any), reinterpret_cast<bf16x8_any *>(p));
}

template <class T>
__global__ __launch_bounds__(kThreads) void state_values(Table a) {
    uint32_t chunk;
    const Tensor &t = find(a, chunk);
    const uint64_t lo = uint64_t(chunk) * a.chunk, hi = min(t.n, lo + a.chunk);
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint8_t *m = static_cast<const uint8_t *>(t.m), *v = static_cast<const uint8_t *>(t.v);
    T *mo = static_cast<T *>(t.w), *vo = reinterpret_cast<T *>(t.master);
    for (uint64_t at = lo + 512 * wave; at < hi; at += 512 * (kThreads / 64)) {
        const uint64_t i = at + 8 * lane;
        if (at + 512 <= hi) {
            const u32x2_any mc = __builtin_nontemporal_load(reinterpret_cast<const u32x2_any *>(m + i));
            const u32x2_any vc = __builtin_nontemporal_load(reinterpret_cast<const u32x2_any *>(v + i));
            const float ms = t.m_scale[i / DF11_ADAMW_BLOCK], vs = t.v_scale[i / DF11_ADAMW_BLOCK];
            f32x4 m0, m1, v0, v1;
            decode(mc[0], vc[0], ms, vs, m0, v0);
            decode(mc[1], vc[1], ms, vs, m1, v1);
            if (mo) store8(mo + i, __builtin_shufflevector(m0, m1, 0, 1, 2, 3, 4, 5, 6, 7));
            if (vo) store8(vo + i, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            for (uint64_t e = i; e < min(i + 8, hi); e++) {
                f32x4 mv, vv;
                decode(m[e], v[e], t.m_scale[e / DF11_ADAMW_BLOCK], t.v_scale[e / DF11_ADAMW_BLOCK], mv, vv);
                if (mo) mo[e] = T(mv[0]);
                if (vo) vo[e] = T(vv[0]);
            }
        }
    }
}

// ---------------------------------------------------------------- gradient norm

// The sum of the workgroup's x, in thread 0, in a fixed order.
template <uint32_t THREADS>
__device__ __forceinline__ double block_sum(double x, double *part) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_down(x, d, 64);
    if ((threadIdx.x & 63u) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    x = part[0];
#pragma unroll
    for (uint32_t p = 1; p < THREADS / 64; p++) x += part[p];
    return x;
}

// Squares of float32 values and their sums in float64: exact squares, no
// overflow, and the fp64 units keep up with HBM.
__device__ __forceinline__ void add_squares(double &s, f32x4 x) {
#pragma unroll
    for (int k = 0; k < 4; k++) s = __builtin_fma(double(x[k]), double(x[k]), s);
}

__device__ __forceinline__ void put_norm(double s, double max_norm, float *out) {
    const double norm = sqrt(s);
    const double f = max_norm / (norm + 1e-6);
    out[0] = float(norm);
    out[1] = norm < __builtin_inf() ? float(f < 1.0 ? f : 1.0) : __builtin_nanf("");
}

// One partial sum per chunk.
template <class G>
__global__ __launch_bounds__(kThreads) void norm_parts(Table a, double *out) {
    __shared__ double part[kThreads / 64];
    uint32_t chunk;
    const Tensor &t = find(a, chunk);
    const uint64_t lo = uint64_t(chunk) * a.chunk, hi = min(t.n, lo + a.chunk);
    const G *g = static_cast<const G *>(t.g);
    const uint32_t i = (threadIdx.x & 63u) * 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    double s = 0.0;
    uint64_t at = lo + 256 * wave;
    for (; at + 3 * kStep + 256 <= hi; at += 4 * kStep) {  // four loads in flight
        f32x4 x[4];
#pragma unroll
        for (int k = 0; k < 4; k++) x[k] = load4<true>(g + at + k * kStep, i, 256);
#pragma unroll
        for (int k = 0; k < 4; k++) add_squares(s, x[k]);
    }
    for (; at < hi; at += kStep)
        add_squares(s, load4<false>(g + at, i, uint32_t(min(hi - at, uint64_t(256)))));
    s = block_sum<kThreads>(s, part);
    if (threadIdx.x == 0) out[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void norm_total(const double *p, uint32_t n, double max_norm,
                                                       float *out) {
    __shared__ double part[kThreads / 64];
    double s = 0.0;
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) s += p[i];
    s = block_sum<kThreads>(s, part);
    if (threadIdx.x == 0) put_norm(s, max_norm, out);
}

// Few elements: one workgroup, whose waves take the chunks (of kOneChunk
// elements) in turn, eight at once, and one launch instead of two: calls one
// behind another 10.5 -> 7.6 us, one alone 19.7 -> 17.6 us; at 65536 elements 20
// us alone by either form, at 131072 24 us.  (A search of the table by scalar
// comparisons took 2 us of it.)
constexpr uint32_t kOneThreads = 1024, kOneWaves = kOneThreads / 64, kOneChunk = 256;
constexpr uint64_t kOneElements = 65536;
constexpr uint32_t kInFlight = 8;

template <class G>
__global__ __launch_bounds__(kOneThreads) void norm_one(Table a, uint32_t chunks, double max_norm,
                                                        float *out) {
    __shared__ double part[kOneWaves];
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t first = lane < kMaxTensors ? a.first[lane] : 0xFFFFFFFFu;
    double s = 0.0;
    for (uint32_t c = wave; c < chunks; c += kInFlight * kOneWaves) {
        f32x4 x[kInFlight];
#pragma unroll
        for (uint32_t k = 0; k < kInFlight; k++) {
            const uint32_t at = c + k * kOneWaves;
            x[k] = f32x4{0, 0, 0, 0};
            if (at >= chunks) continue;
            const uint32_t j = __popcll(__builtin_amdgcn_ballot_w64(at >= first)) - 1;  // its tensor
            const uint32_t lo = (at - a.first[j]) * kOneChunk, left = uint32_t(a.t[j].n) - lo;
            const G *g = static_cast<const G *>(a.t[j].g) + lo;
            x[k] = left >= kOneChunk ? load4<true>(g, 4 * lane, left) : load4<false>(g, 4 * lane, left);
        }
#pragma unroll
        for (uint32_t k = 0; k < kInFlight; k++) add_squares(s, x[k]);
    }
    s = block_sum<kOneThreads>(s, part);
    if (threadIdx.x == 0) put_norm(s, max_norm, out);
}

// ---------------------------------------------------------------- host

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

uint64_t total(const df11_adamw_tensor *t, uint32_t n) {
    uint64_t s = 0;
    for (uint32_t k = 0; k < n; k++) s += t[k].numel;
    return s;
}

// Elements per workgroup: as many as leave about `groups` workgroups, between
// one iteration and `most`; more where a tensor would have 2^23 chunks (a grid
// holds less than 2^32 threads).
constexpr uint32_t kMaxChunks = (1u << 24) - 1;
uint32_t chunk_for(const df11_adamw_tensor *t, uint32_t n, uint64_t groups, uint32_t most) {
    const uint64_t elements = total(t, n);
    uint64_t longest = 0;
    for (uint32_t k = 0; k < n; k++) longest = t[k].numel > longest ? t[k].numel : longest;
    uint32_t c = kStep;
    while ((c < most && elements / c > groups) || (c < 1u << 30 && longest / c >= 1u << 23)) c *= 2;
    return c;
}

// Fills tables with the tensors that are not empty and runs each: run(table, its chunks, its tensors)
template <class Fill, class Run>
int each_table(const df11_adamw_tensor *t, uint32_t n, uint32_t chunk, Fill fill, Run run) {
    uint32_t k = 0;
    while (k < n) {
        Table a{};
        a.chunk = chunk;
        for (uint32_t &f : a.first) f = 0xFFFFFFFFu;
        uint64_t chunks = 0;
        uint32_t used = 0;
        for (; k < n && used < kMaxTensors; k++) {
            if (!t[k].numel) continue;
            const uint64_t more = (t[k].numel + chunk - 1) / chunk;
            if (chunks + more > kMaxChunks) break;
            a.first[used] = uint32_t(chunks);
            a.t[used].n = t[k].numel;
            fill(a.t[used], k);
            chunks += more;
            used++;
        }
        if (used) {
            const int rc = run(a, uint32_t(chunks), used);
            if (rc != DF11_OK) return rc;
        }
    }
    return DF11_OK;
}

int status(hipError_t e) { return e == hipSuccess ? DF11_OK : DF11_E_HIP; }

template <class W, bool MASTER, class G, int BITS, bool COUNTS>
int run_step(const Table &a, uint32_t grid, const Numbers &c, hipStream_t st) {
    return status(launch(adamw<W, MASTER, G, BITS, COUNTS>, dim3(grid), dim3(kThreads), 0, st, a, c));
}

template <class W, bool MASTER, bool COUNTS>
int pick_step(const Table &a, uint32_t grid, const Numbers &c, hipStream_t st, bool g16, bool s8) {
    if (g16)
        return s8 ? run_step<W, MASTER, __bf16, 8, COUNTS>(a, grid, c, st)
                  : run_step<W, MASTER, __bf16, 32, COUNTS>(a, grid, c, st);
    return s8 ? run_step<W, MASTER, float, 8, COUNTS>(a, grid, c, st)
              : run_step<W, MASTER, float, 32, COUNTS>(a, grid, c, st);
}

bool finite_at_least_0(double x) { return std::isfinite(x) && x >= 0.0; }

// The step; d_skipped and d_count as in Numbers.
int adamw_step(const df11_adamw_config *c, const df11_adamw_tensor *t, uint32_t n_tensors,
               const uint64_t *d_skipped, uint64_t *d_count, uint64_t more, hipStream_t st) {
    if (!c || (n_tensors && !t)) return DF11_E_INVALID;
    if (c->w_type > DF11_TYPE_BF16 || c->g_type > DF11_TYPE_BF16 || c->reserved ||
        (c->state_bits != 32 && c->state_bits != 8))
        return DF11_E_INVALID;
    const auto is_beta = [](double b) { return b >= 0.0 && b < 1.0; };
    if (!finite_at_least_0(c->lr) || !is_beta(c->beta1) || !is_beta(c->beta2) ||
        !std::isfinite(c->eps) || !(float(c->eps) > 0.0f) || (!c->d_step && c->step < 1))
        return DF11_E_INVALID;
    if (!aligned(c->d_lr, 4) || !aligned(c->d_step, 8) || !aligned(c->d_grad_factor, 4))
        return DF11_E_INVALID;
    const bool w16 = c->w_type == DF11_TYPE_BF16, g16 = c->g_type == DF11_TYPE_BF16;
    const bool s8 = c->state_bits == 8;
    const uintptr_t state_size = s8 ? 1 : 4;
    bool masters = false, plain = false, counts = false;
    uint32_t last = 0;  // the last tensor that is not empty: its launch is the call's last
    for (uint32_t k = 0; k < n_tensors; k++) {
        const df11_adamw_tensor &x = t[k];
        if (x.numel > kMaxNumel || !finite_at_least_0(x.lr_scale) ||
            !finite_at_least_0(x.weight_decay))
            return DF11_E_INVALID;
        if ((x.master || x.counts) && !w16) return DF11_E_INVALID;
        if (!aligned(x.counts, 8)) return DF11_E_INVALID;
        counts = counts || x.counts;
        if (!x.numel) continue;
        if (!x.w || !x.g || !x.m || !x.v || (s8 && (!x.m_scale || !x.v_scale))) return DF11_E_INVALID;
        if (!aligned(x.w, w16 ? 2 : 4) || !aligned(x.g, g16 ? 2 : 4) || !aligned(x.m, state_size) ||
            !aligned(x.v, state_size) || !aligned(x.master, 4) || !aligned(x.m_scale, 4) ||
            !aligned(x.v_scale, 4))
            return DF11_E_INVALID;
        (x.master ? masters : plain) = true;
        last = k;
    }
    if (masters && plain) return DF11_E_INVALID;  // one kernel serves all tensors

    Numbers num{};
    const double step = double(c->step);
    num.b1 = float(c->beta1), num.c1 = float(1.0 - c->beta1);
    num.b2 = float(c->beta2), num.c2 = float(1.0 - c->beta2);
    num.eps = float(c->eps);
    num.bias1 = 1.0 - std::pow(c->beta1, step);
    num.inv_root = float(1.0 / std::sqrt(1.0 - std::pow(c->beta2, step)));
    num.lr = c->lr;
    num.log_b1 = std::log(c->beta1), num.log_b2 = std::log(c->beta2);
    num.d_lr = c->d_lr, num.d_step = c->d_step, num.d_factor = c->d_grad_factor;
    num.step = c->step, num.d_skipped = d_skipped, num.more = more;

    const auto fill = [&](Tensor &a, uint32_t k) {
        const df11_adamw_tensor &x = t[k];
        if (k == last) num.d_count = reinterpret_cast<unsigned long long *>(d_count);
        a.w = x.w, a.master = x.master, a.g = x.g, a.m = x.m, a.v = x.v;
        a.m_scale = x.m_scale, a.v_scale = x.v_scale;
        a.counts = reinterpret_cast<unsigned long long *>(x.counts);
        const double lr = c->lr * x.lr_scale;
        a.keep = float(1.0 - lr * x.weight_decay);
        a.size = float(lr / num.bias1);
        a.lr_scale = x.lr_scale, a.weight_decay = x.weight_decay;
    };
    if (counts) {  // all of them before the first weight is counted: tensors may share an array
        for (uint32_t k = 0; k < n_tensors;) {
            Table a{};
            uint32_t used = 0;
            for (; k < n_tensors && used < kMaxTensors; k++)
                if (t[k].counts) a.t[used++].counts = reinterpret_cast<unsigned long long *>(t[k].counts);
            if (used && launch(clear_counts, dim3(used), dim3(256), 0, st, a) != hipSuccess)
                return DF11_E_HIP;
        }
    }
    return each_table(t, n_tensors, chunk_for(t, n_tensors, 2048, 8 * kStep), fill,
                      [&](const Table &a, uint32_t grid, uint32_t) {
                          if (!w16) return pick_step<float, false, false>(a, grid, num, st, g16, s8);
                          if (masters)
                              return counts ? pick_step<__bf16, true, true>(a, grid, num, st, g16, s8)
                                            : pick_step<__bf16, true, false>(a, grid, num, st, g16, s8);
                          return counts ? pick_step<__bf16, false, true>(a, grid, num, st, g16, s8)
                                        : pick_step<__bf16, false, false>(a, grid, num, st, g16, s8);
                      });
}

}  // namespace

extern "C" {

int df11_adamw_step(const df11_adamw_config *c, const df11_adamw_tensor *t, uint32_t n_tensors,
                    df11_hip_stream stream) {
    return adamw_step(c, t, n_tensors, nullptr, nullptr, 0, static_cast<hipStream_t>(stream));
}

int df11_adamw_step_counted(const df11_adamw_config *c, const df11_adamw_tensor *t, uint32_t n_tensors,
                            uint64_t *d_count, df11_hip_stream stream) {
    if (!c || !d_count || !aligned(d_count, 8) || (c->d_step && c->d_step != d_count)) return DF11_E_INVALID;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return c->d_step ? adamw_step(c, t, n_tensors, nullptr, d_count, ~uint64_t(0), st)  // one less
                     : adamw_step(c, t, n_tensors, d_count, d_count, 1, st);
}

int df11_adamw_values(const df11_adamw_tensor *t, uint32_t n_tensors, uint32_t type,
                      void *const *m_out, void *const *v_out, df11_hip_stream stream) {
    hipStream_t st = static_cast<hipStream_t>(stream);
    if ((n_tensors && !t) || type > DF11_TYPE_BF16) return DF11_E_INVALID;
    const uintptr_t size = type == DF11_TYPE_BF16 ? 2 : 4;
    for (uint32_t k = 0; k < n_tensors; k++) {
        if (t[k].numel > kMaxNumel) return DF11_E_INVALID;
        if (!t[k].numel) continue;
        if (!t[k].m || !t[k].v || !t[k].m_scale || !t[k].v_scale || !aligned(t[k].m_scale, 4) ||
            !aligned(t[k].v_scale, 4))
            return DF11_E_INVALID;
        if ((m_out && (!m_out[k] || !aligned(m_out[k], size))) ||
            (v_out && (!v_out[k] || !aligned(v_out[k], size))))
            return DF11_E_INVALID;
    }
    const auto fill = [&](Tensor &a, uint32_t k) {
        a.m = t[k].m, a.v = t[k].v, a.m_scale = t[k].m_scale, a.v_scale = t[k].v_scale;
        a.w = m_out ? m_out[k] : nullptr;
        a.master = v_out ? static_cast<float *>(v_out[k]) : nullptr;
    };
    return each_table(t, n_tensors, chunk_for(t, n_tensors, 2048, 8 * kStep), fill,
                      [&](const Table &a, uint32_t grid, uint32_t) {
                          return status(type == DF11_TYPE_BF16
                                            ? launch(state_values<__bf16>, dim3(grid), dim3(kThreads), 0, st, a)
                                            : launch(state_values<float>, dim3(grid), dim3(kThreads), 0, st, a));
                      });
}

uint64_t df11_grad_norm_scratch_bytes(const df11_adamw_tensor *t, uint32_t n_tensors) {
    if (!t) return 8;
    const uint32_t chunk = chunk_for(t, n_tensors, 4096, 64 * kStep);
    uint64_t parts = 0;
    for (uint32_t k = 0; k < n_tensors; k++) parts += (t[k].numel + chunk - 1) / chunk;
    return 8 * (parts ? parts : 1);
}

int df11_grad_norm(uint32_t g_type, const df11_adamw_tensor *t, uint32_t n_tensors, double max_norm,
                   float *d_norm, void *scratch, uint64_t scratch_bytes, df11_hip_stream stream) {
    hipStream_t st = static_cast<hipStream_t>(stream);
    if ((n_tensors && !t) || g_type > DF11_TYPE_BF16 || !(max_norm > 0.0) || !d_norm ||
        !aligned(d_norm, 4) || !scratch || !aligned(scratch, 8))
        return DF11_E_INVALID;
    const bool g16 = g_type == DF11_TYPE_BF16;
    for (uint32_t k = 0; k < n_tensors; k++) {
        if (t[k].numel > kMaxNumel) return DF11_E_INVALID;
        if (t[k].numel && (!t[k].g || !aligned(t[k].g, g16 ? 2 : 4))) return DF11_E_INVALID;
    }
    if (scratch_bytes < df11_grad_norm_scratch_bytes(t, n_tensors)) return DF11_E_INVALID;
    uint32_t used = 0;
    for (uint32_t k = 0; k < n_tensors; k++) used += t[k].numel != 0;
    if (used && used <= kMaxTensors && total(t, n_tensors) <= kOneElements)
        return each_table(
            t, n_tensors, kOneChunk, [&](Tensor &a, uint32_t k) { a.g = t[k].g; },
            [&](const Table &a, uint32_t chunks, uint32_t) {
                return status(g16 ? launch(norm_one<__bf16>, dim3(1), dim3(kOneThreads), 0, st, a, chunks,
                                           max_norm, d_norm)
                                  : launch(norm_one<float>, dim3(1), dim3(kOneThreads), 0, st, a, chunks,
                                           max_norm, d_norm));
            });
    double *parts = static_cast<double *>(scratch);
    uint64_t done = 0;
    const int rc = each_table(
        t, n_tensors, chunk_for(t, n_tensors, 4096, 64 * kStep),
        [&](Tensor &a, uint32_t k) { a.g = t[k].g; },
        [&](const Table &a, uint32_t grid, uint32_t) {
            double *p = parts + done;
            done += grid;
            return status(g16 ? launch(norm_parts<__bf16>, dim3(grid), dim3(kThreads), 0, st, a, p)
                              : launch(norm_parts<float>, dim3(grid), dim3(kThreads), 0, st, a, p));
        });
    if (rc != DF11_OK) return rc;
    if (done > 0xFFFFFFFFu) return DF11_E_INVALID;
    return status(launch(norm_total, dim3(1), dim3(kThreads), 0, st,
                         static_cast<const double *>(parts), uint32_t(done), max_norm, d_norm));
}

}  // extern "C"
