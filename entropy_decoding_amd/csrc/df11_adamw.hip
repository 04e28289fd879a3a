// AdamW over many tensors, the gradients' norm, and the reader of 8-bit states.
//
// A step is one pass over the tensors: every element's gradient, weight and
// states are read once and written once, so HBM bounds it.  A workgroup takes
// a chunk of one tensor; the table that says which one travels in the kernel
// arguments, so a call needs no device memory of its own.  A wave works on
// 256 consecutive elements at a time, 4 a lane: every access of a wave is
// contiguous, and 256 elements are one block of 8-bit states, whose largest
// values are a reduction inside the wave.
//
// Contraction is off: each product and sum is rounded on its own, so that a
// weight does not depend on how the compiler pairs them and an elementwise
// implementation in float32 gives the same bits.
#include <hip/hip_runtime.h>

#include <cmath>

#include "df11.h"
#include "df11_launch.h"

#pragma clang fp contract(off)

namespace {

using df11_detail::launch;

constexpr uint32_t kThreads = 256;
constexpr uint32_t kStep = kThreads * 4;    // elements of a workgroup's iteration
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
};

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32_any __attribute__((aligned(1)));

// 4 elements at p[i ..], zeros from n on; the hardware takes any alignment
__device__ __forceinline__ f32x4 load4(const float *p, uint64_t i, uint64_t n) {
    if (i + 4 <= n) return *reinterpret_cast<const f32x4_any *>(p + i);
    f32x4 x = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 3; k++)
        if (i + k < n) x[k] = p[i + k];
    return x;
}
__device__ __forceinline__ f32x4 load4(const __bf16 *p, uint64_t i, uint64_t n) {
    if (i + 4 <= n)
        return __builtin_convertvector(*reinterpret_cast<const bf16x4_any *>(p + i), f32x4);
    f32x4 x = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 3; k++)
        if (i + k < n) x[k] = float(p[i + k]);
    return x;
}
__device__ __forceinline__ uint32_t load4(const uint8_t *p, uint64_t i, uint64_t n) {
    if (i + 4 <= n) return *reinterpret_cast<const u32_any *>(p + i);
    uint32_t x = 0;
#pragma unroll
    for (int k = 0; k < 3; k++)
        if (i + k < n) x |= uint32_t(p[i + k]) << (8 * k);
    return x;
}
__device__ __forceinline__ void store4(float *p, uint64_t i, uint64_t n, f32x4 x) {
    if (i + 4 <= n) {
        *reinterpret_cast<f32x4_any *>(p + i) = x;
        return;
    }
#pragma unroll
    for (int k = 0; k < 3; k++)
        if (i + k < n) p[i + k] = x[k];
}
__device__ __forceinline__ void store4(__bf16 *p, uint64_t i, uint64_t n, bf16x4 x) {
    if (i + 4 <= n) {
        *reinterpret_cast<bf16x4_any *>(p + i) = x;
        return;
    }
#pragma unroll
    for (int k = 0; k < 3; k++)
        if (i + k < n) p[i + k] = x[k];
}
__device__ __forceinline__ void store4(__bf16 *p, uint64_t i, uint64_t n, f32x4 x) {
    store4(p, i, n, __builtin_convertvector(x, bf16x4));
}
__device__ __forceinline__ void store4(uint8_t *p, uint64_t i, uint64_t n, uint32_t x) {
    if (i + 4 <= n) {
        *reinterpret_cast<u32_any *>(p + i) = x;
        return;
    }
#pragma unroll
    for (int k = 0; k < 3; k++)
        if (i + k < n) p[i + k] = uint8_t(x >> (8 * k));
}

// the largest x of the wave, in every lane (DPP inside rows of 16, then across rows)
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x111, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x112, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x114, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x118, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x142, 0xF, 0xF, false)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x143, 0xF, 0xF, false)));
    return uint32_t(__builtin_amdgcn_readlane(int(x), 63));
}

// The scale of a block from the bits of its largest magnitude (magnitudes
// compare as their bits do, and NaN above all), and its reciprocal.
// unit = 1 / 127^2 or 1 / 255^2, rounded.
__device__ __forceinline__ void block_scale(uint32_t top, float unit, float tiny, float &scale,
                                            float &inv) {
    const float x = __uint_as_float(top);
    const bool bad = top >= 0x7F800000u;
    const bool none = x < tiny;
    scale = bad ? __uint_as_float(0x7FC00000u) : none ? 0.0f : x * unit;
    inv = bad || none ? 0.0f : 1.0f / scale;
}

__device__ __forceinline__ const Tensor &find(const Table &a, uint32_t &chunk) {
    uint32_t k = 0;
#pragma unroll
    for (uint32_t j = 1; j < kMaxTensors; j++) k += uint32_t(blockIdx.x >= a.first[j]);
    chunk = blockIdx.x - a.first[k];
    return a.t[k];
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

    float keep = t.keep, size = t.size, inv_root = c.inv_root, f = 1.0f;
    if (c.d_lr || c.d_step) {
        const double lr = (c.d_lr ? double(*c.d_lr) : c.lr) * t.lr_scale;
        double bias1 = c.bias1;
        if (c.d_step) {
            const double step = double(*c.d_step);
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
    }

    W *w = static_cast<W *>(t.w);
    const G *g = static_cast<const G *>(t.g);
    for (uint64_t i = lo + threadIdx.x * 4; i < ((hi + 255) & ~uint64_t(255)); i += kStep) {
        bf16x4 shown;  // the weights as BF16, for the histogram
        if (still) {
            if (!counting) break;
            shown = __builtin_convertvector(load4(w, i, hi), bf16x4);
        } else {
            const uint64_t b = i / DF11_ADAMW_BLOCK;  // the same in all lanes of a wave
            f32x4 gr = load4(g, i, hi);
            f32x4 x = MASTER ? load4(t.master, i, hi) : load4(w, i, hi);
            f32x4 m, v;
            if constexpr (BITS == 32) {
                m = load4(static_cast<const float *>(t.m), i, hi);
                v = load4(static_cast<const float *>(t.v), i, hi);
            } else {
                const uint32_t mc = load4(static_cast<const uint8_t *>(t.m), i, hi);
                const uint32_t vc = load4(static_cast<const uint8_t *>(t.v), i, hi);
                const float ms = t.m_scale[b], vs = t.v_scale[b];
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const int cm = int(int8_t(mc >> (8 * k)));
                    const int cv = int(uint8_t(vc >> (8 * k)));
                    m[k] = ms * float(cm * (cm < 0 ? -cm : cm));
                    const float r = vs * float(cv * cv);
                    v[k] = r * r;
                }
            }
            f32x4 r;
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const float gk = c.d_factor ? gr[k] * f : gr[k];
                m[k] = m[k] * c.b1 + gk * c.c1;
                v[k] = v[k] * c.b2 + (gk * c.c2) * gk;
                r[k] = sqrtf(v[k]);
                const float u = m[k] / (r[k] * inv_root + c.eps);
                x[k] = x[k] * keep - u * size;
            }
            if constexpr (BITS == 32) {
                store4(static_cast<float *>(t.m), i, hi, m);
                store4(static_cast<float *>(t.v), i, hi, v);
            } else {
                uint32_t tm = 0, tr = 0;
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    if (i + k >= hi) m[k] = r[k] = 0.0f;
                    tm = max(tm, __float_as_uint(m[k]) & 0x7FFFFFFFu);
                    tr = max(tr, __float_as_uint(r[k]) & 0x7FFFFFFFu);
                }
                float ms, mi, vs, vi;
                block_scale(wave_max(tm), 1.0f / (127.0f * 127.0f), 0x1p-100f, ms, mi);
                block_scale(wave_max(tr), 1.0f / (255.0f * 255.0f), 0x1p-149f, vs, vi);
                uint32_t mc = 0, vc = 0;
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const int cm = int(fminf(rintf(sqrtf(fabsf(m[k]) * mi)), 127.0f));
                    int cv = int(fminf(rintf(sqrtf(r[k] * vi)), 255.0f));
                    if (vi > 0.0f && r[k] > 0.0f) cv = max(cv, 1);
                    mc |= (uint32_t(m[k] < 0.0f ? -cm : cm) & 0xFFu) << (8 * k);
                    vc |= uint32_t(cv) << (8 * k);
                }
                store4(static_cast<uint8_t *>(t.m), i, hi, mi > 0.0f ? mc : 0u);
                store4(static_cast<uint8_t *>(t.v), i, hi, vi > 0.0f ? vc : 0u);
                if ((threadIdx.x & 63u) == 0) {
                    t.m_scale[b] = ms;
                    t.v_scale[b] = vs;
                }
            }
            if (MASTER) store4(t.master, i, hi, x);
            if constexpr (sizeof(W) == 2) {
                shown = __builtin_convertvector(x, bf16x4);
                store4(w, i, hi, shown);
            } else {
                store4(w, i, hi, x);
            }
        }
        if (counting) {
            const uint32_t copy = threadIdx.x % kCopies;
            const uint16_t *bits = reinterpret_cast<const uint16_t *>(&shown);
#pragma unroll
            for (int k = 0; k < 4; k++)
                if (i + k < hi)
                    atomicAdd(&hist[((bits[k] >> 7) & 0xFFu) * (kCopies + 1) + copy], 1u);
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

// m and v of 8-bit states; the outputs travel in the table's w and master
template <class T>
__global__ __launch_bounds__(kThreads) void state_values(Table a) {
    uint32_t chunk;
    const Tensor &t = find(a, chunk);
    const uint64_t lo = uint64_t(chunk) * a.chunk, hi = min(t.n, lo + a.chunk);
    T *mo = static_cast<T *>(t.w), *vo = reinterpret_cast<T *>(t.master);
    for (uint64_t i = lo + threadIdx.x * 4; i < hi; i += kStep) {
        const uint64_t b = i / DF11_ADAMW_BLOCK;
        f32x4 m, v;
        const uint32_t mc = load4(static_cast<const uint8_t *>(t.m), i, hi);
        const uint32_t vc = load4(static_cast<const uint8_t *>(t.v), i, hi);
        const float ms = t.m_scale[b], vs = t.v_scale[b];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int cm = int(int8_t(mc >> (8 * k)));
            const int cv = int(uint8_t(vc >> (8 * k)));
            m[k] = ms * float(cm * (cm < 0 ? -cm : cm));
            const float r = vs * float(cv * cv);
            v[k] = r * r;
        }
        if (mo) store4(mo, i, hi, m);
        if (vo) store4(vo, i, hi, v);
    }
}

// ---------------------------------------------------------------- gradient norm

// The sum of the workgroup's x, in thread 0, in a fixed order.
__device__ __forceinline__ double block_sum(double x, double *part) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_down(x, d, 64);
    if ((threadIdx.x & 63u) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    return part[0] + part[1] + part[2] + part[3];
}

// One partial sum per chunk.  Squares of float32 values and their sums in
// float64: exact squares, no overflow, and the fp64 units keep up with HBM.
template <class G>
__global__ __launch_bounds__(kThreads) void norm_parts(Table a, double *out) {
    __shared__ double part[kThreads / 64];
    uint32_t chunk;
    const Tensor &t = find(a, chunk);
    const uint64_t lo = uint64_t(chunk) * a.chunk, hi = min(t.n, lo + a.chunk);
    const G *g = static_cast<const G *>(t.g);
    double s = 0.0;
    for (uint64_t i = lo + threadIdx.x * 4; i < hi; i += kStep) {
        const f32x4 x = load4(g, i, hi);
#pragma unroll
        for (int k = 0; k < 4; k++) s = __builtin_fma(double(x[k]), double(x[k]), s);
    }
    s = block_sum(s, part);
    if (threadIdx.x == 0) out[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void norm_total(const double *p, uint32_t n, double max_norm,
                                                       float *out) {
    __shared__ double part[kThreads / 64];
    double s = 0.0;
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) s += p[i];
    s = block_sum(s, part);
    if (threadIdx.x == 0) {
        const double norm = sqrt(s);
        const double f = max_norm / (norm + 1e-6);
        out[0] = float(norm);
        out[1] = norm < __builtin_inf() ? float(f < 1.0 ? f : 1.0) : __builtin_nanf("");
    }
}

// ---------------------------------------------------------------- host

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

uint64_t total(const df11_adamw_tensor *t, uint32_t n) {
    uint64_t s = 0;
    for (uint32_t k = 0; k < n; k++) s += t[k].numel;
    return s;
}

// Elements per workgroup: as many as leave about `groups` workgroups, between
// one iteration and `most`.
uint32_t chunk_for(uint64_t elements, uint64_t groups, uint32_t most) {
    uint32_t c = kStep;
    while (c < most && elements / c > groups) c *= 2;
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
            if (chunks + more > 0x7FFFFFFFu) break;
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

}  // namespace

extern "C" {

int df11_adamw_step(const df11_adamw_config *c, const df11_adamw_tensor *t, uint32_t n_tensors,
                    df11_hip_stream stream) {
    hipStream_t st = static_cast<hipStream_t>(stream);
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

    const auto fill = [&](Tensor &a, uint32_t k) {
        const df11_adamw_tensor &x = t[k];
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
    return each_table(t, n_tensors, chunk_for(total(t, n_tensors), 2048, 8 * kStep), fill,
                      [&](const Table &a, uint32_t grid, uint32_t) {
                          if (!w16) return pick_step<float, false, false>(a, grid, num, st, g16, s8);
                          if (masters)
                              return counts ? pick_step<__bf16, true, true>(a, grid, num, st, g16, s8)
                                            : pick_step<__bf16, true, false>(a, grid, num, st, g16, s8);
                          return counts ? pick_step<__bf16, false, true>(a, grid, num, st, g16, s8)
                                        : pick_step<__bf16, false, false>(a, grid, num, st, g16, s8);
                      });
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
    return each_table(t, n_tensors, chunk_for(total(t, n_tensors), 2048, 8 * kStep), fill,
                      [&](const Table &a, uint32_t grid, uint32_t) {
                          return status(type == DF11_TYPE_BF16
                                            ? launch(state_values<__bf16>, dim3(grid), dim3(kThreads), 0, st, a)
                                            : launch(state_values<float>, dim3(grid), dim3(kThreads), 0, st, a));
                      });
}

uint64_t df11_grad_norm_scratch_bytes(const df11_adamw_tensor *t, uint32_t n_tensors) {
    if (!t) return 8;
    const uint32_t chunk = chunk_for(total(t, n_tensors), 4096, 64 * kStep);
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
    double *parts = static_cast<double *>(scratch);
    uint64_t done = 0;
    const int rc = each_table(
        t, n_tensors, chunk_for(total(t, n_tensors), 4096, 64 * kStep),
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
