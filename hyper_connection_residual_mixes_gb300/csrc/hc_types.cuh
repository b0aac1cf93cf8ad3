// hc_types.cuh -- runs of fp32, bf16 or fp16 values as the sublayer operators
// hold them: one element, a vector, or pairs for the packed fp32 instructions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "hc_device.cuh"

namespace hc {

template <typename T>
__device__ __forceinline__ float to_f(T v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (__is_same(T, __half)) return __half2float(v);
    else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f(float v) {  // to nearest, ties to even
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (__is_same(T, __half)) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};
template <typename T, int V>
union Words {  // the same in 32-bit words
    Vec<T, V> v;
    uint32_t w[sizeof(T) * V / 4];
};

// values k, k + 1 (k even) as an fp32 pair, and back
template <typename T, int V>
__device__ __forceinline__ f32x2 pair(const Vec<T, V> &x, int k) {
    if constexpr (sizeof(T) == 4) {
        return f2_make(x.v[k], x.v[k + 1]);
    } else {
        Words<T, V> u;
        u.v = x;
        if constexpr (__is_same(T, __half)) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u.w[k / 2]));
            return f2_make(f.x, f.y);
        } else {
            return f2_from_bf16x2(u.w[k / 2]);
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ void put_pair(Vec<T, V> &x, int k, f32x2 v) {
    float a, b;
    f2_split(v, a, b);
    if constexpr (sizeof(T) == 4) {
        x.v[k] = a, x.v[k + 1] = b;
    } else {
        Words<T, V> u;
        u.v = x;
        if constexpr (__is_same(T, __half)) {
            const __half2 h = __floats2half2_rn(a, b);
            u.w[k / 2] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            u.w[k / 2] = pack_bf16x2(a, b);
        }
        x = u.v;
    }
}

}  // namespace hc
