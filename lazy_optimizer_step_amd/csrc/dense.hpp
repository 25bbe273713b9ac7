// dense.hpp - what the dense operators' sources share.
#pragma once

#include "common.hpp"
#include "dense_ops.h"

namespace spopt {

inline size_t dtype_bytes(int32_t dtype) { return dtype == SPOPT_DTYPE_F32 ? 4 : 2; }

// V values at p, which need only be aligned to one of them: gfx950 takes
// 16-byte global accesses at any address, and rows of odd widths or strides
// start anywhere.
template <class T, int V>
struct Pack {
    typedef T type __attribute__((ext_vector_type(V), aligned(sizeof(T))));
};
template <class T>
struct Pack<T, 1> {
    typedef T type;
};

template <class T, int V>
__device__ __forceinline__ void load_v(const T* p, float (&x)[V]) {
    const auto q = *reinterpret_cast<const typename Pack<T, V>::type*>(p);
    if constexpr (V == 1)
        x[0] = (float)q;
    else
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = (float)q[e];
}

template <class T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&x)[V]) {
    typename Pack<T, V>::type q;
    if constexpr (V == 1)
        q = (T)x[0];
    else
#pragma unroll
        for (int e = 0; e < V; ++e) q[e] = (T)x[e];
    *reinterpret_cast<typename Pack<T, V>::type*>(p) = q;
}

// Sets kStatusNonFinite where a rows x cols array (row stride in elements)
// holds a NaN or an infinity.
int launch_check_finite(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride,
                        uint32_t* status, hipStream_t s);

}  // namespace spopt
