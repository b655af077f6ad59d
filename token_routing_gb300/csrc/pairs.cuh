// Sixteen bytes of elements as packed fp32 pairs, and back (training-step kernels).
#pragma once

#include "internal.cuh"

namespace moe {

// The 16 bytes of a vector as fp32 pairs.
template <typename T> struct Pairs { static constexpr int N = 8 / sizeof(T); };
template <typename T>
__device__ __forceinline__ void to_pairs(const uint4& u, uint64_t (&p)[Pairs<T>::N]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = pk2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
        p[0] = pk2(__uint_as_float(w[0]), __uint_as_float(w[1]));
        p[1] = pk2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    }
}
template <typename T>
__device__ __forceinline__ uint4 from_pairs(const uint64_t (&p)[Pairs<T>::N]) {
    uint32_t w[4];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            upk2(p[i], lo, hi);
            const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    } else {
        float f[4];
        upk2(p[0], f[0], f[1]);
        upk2(p[1], f[2], f[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(f[i]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace moe
