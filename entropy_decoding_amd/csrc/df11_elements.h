// Elements of the operators' tensors in groups of eight, at any alignment, as
// float32.
#pragma once

#include <hip/hip_runtime.h>

#include "df11.h"

#include <cstdint>

namespace df11_detail {

__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// Eight consecutive elements of T that need T's alignment only: gfx950 loads
// and stores 16 bytes at any address.
template <class T>
struct Group {
    typedef T type __attribute__((ext_vector_type(8)));
    typedef type any __attribute__((aligned(sizeof(T))));
};

template <class T>
__device__ __forceinline__ f32x8 widen(typename Group<T>::type v) {
    f32x8 r;
#pragma unroll
    for (int e = 0; e < 8; e++) r[e] = float(v[e]);
    return r;
}

// Columns c .. c + 7 of a row of `cols`; columns past the end are 0.  ONCE: what is
// read once passes the caches by.
template <class T, bool ONCE = false>
__device__ __forceinline__ typename Group<T>::type load_group(const T *row, uint32_t c, uint32_t cols) {
    typedef typename Group<T>::any any;
    if (c + 8 <= cols)
        return ONCE ? __builtin_nontemporal_load(reinterpret_cast<const any *>(row + c))
                    : *reinterpret_cast<const any *>(row + c);
    typename Group<T>::type v;
#pragma unroll
    for (uint32_t e = 0; e < 8; e++) v[e] = c + e < cols ? row[c + e] : T(0.0f);
    return v;
}

// The group rounded to T (to nearest, ties to even) into columns c .. c + 7; PAST the
// caches, or not.
template <class T, bool PAST = false>
__device__ __forceinline__ void store_group(T *row, uint32_t c, uint32_t cols, f32x8 x) {
    typedef typename Group<T>::any any;
    any v;
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = T(x[e]);
    if (c + 8 <= cols) {
        if (PAST) __builtin_nontemporal_store(v, reinterpret_cast<any *>(row + c));
        else *reinterpret_cast<any *>(row + c) = v;
    } else {
#pragma unroll
        for (uint32_t e = 0; e < 7; e++)
            if (c + e < cols) row[c + e] = v[e];
    }
}

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int status(hipError_t e) { return e == hipSuccess ? DF11_OK : DF11_E_HIP; }
inline uint32_t type_bytes(uint32_t type) { return type == DF11_TYPE_F32 ? 4 : 2; }

// f(a value of the C++ type that `type` names)
template <class F>
int with_type(uint32_t type, F f) {
    switch (type) {
    case DF11_TYPE_F32: return f(float{});
    case DF11_TYPE_BF16: return f(__bf16{});
    default: return f(_Float16{});
    }
}

}  // namespace df11_detail
