// two_byte.cuh -- bf16 and fp16 values in registers, eight (16 bytes) at a time.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace topkidx {

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    using two = __nv_bfloat162;
    static __device__ __forceinline__ float2 wide(two x) { return __bfloat1622float2(x); }
    static __device__ __forceinline__ two narrow(float2 x) { return __float22bfloat162_rn(x); }
};
template <>
struct Pair<__half> {
    using two = __half2;
    static __device__ __forceinline__ float2 wide(two x) { return __half22float2(x); }
    static __device__ __forceinline__ two narrow(float2 x) { return __float22half2_rn(x); }
};

template <typename T>
struct alignas(16) Eight {
    typename Pair<T>::two v[4];
};

template <typename T>
__device__ __forceinline__ void widen(const Eight<T>& x, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = Pair<T>::wide(x.v[i]);
        f[2 * i] = y.x;
        f[2 * i + 1] = y.y;
    }
}

template <typename T>
__device__ __forceinline__ Eight<T> narrow(const float* f) {
    Eight<T> x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = Pair<T>::narrow(make_float2(f[2 * i], f[2 * i + 1]));
    return x;
}

}  // namespace topkidx
