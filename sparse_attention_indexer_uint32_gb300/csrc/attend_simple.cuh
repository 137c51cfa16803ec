// attend_simple.cuh -- one query head's attention by one block of four warps:
// the warps take the keys in turn, each with its own running maximum and sum,
// and join at the end.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace topkidx {

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float x) {
    return __float2half_rn(x);
}

constexpr int kSimpleWarps = 4;

// kD / kE: query and value sizes.  key(j, d) and value(j, e) load an element;
// seen(j) says whether key j counts (its loads are not made otherwise).
template <typename T, int kD, int kE, typename Q, typename Seen, typename Key, typename Value>
__device__ void simple_attend(int n, float scale, Q query, Seen seen, Key key, Value value, T* out, float* lse) {
    __shared__ float part[kSimpleWarps][kE];
    __shared__ float part_m[kSimpleWarps], part_l[kSimpleWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float q[kD / 32], o[kE / 32] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < kD / 32; ++i) q[i] = query(lane + 32 * i);
    for (int j = warp; j < n; j += kSimpleWarps) {
        if (!seen(j)) continue;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kD / 32; ++i) s += q[i] * key(j, lane + 32 * i);
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        s *= scale;
        const float top = fmaxf(m, s);
        const float back = m == top ? 1.f : expf(m - top), p = s == top ? 1.f : expf(s - top);
        l = l * back + p;
#pragma unroll
        for (int i = 0; i < kE / 32; ++i) o[i] = o[i] * back + p * value(j, lane + 32 * i);
        m = top;
    }
#pragma unroll
    for (int i = 0; i < kE / 32; ++i) part[warp][lane + 32 * i] = o[i];
    if (lane == 0) {
        part_m[warp] = m;
        part_l[warp] = l;
    }
    __syncthreads();
    float top = -INFINITY, sum = 0.f, by[kSimpleWarps];
    for (int w = 0; w < kSimpleWarps; ++w) top = fmaxf(top, part_m[w]);
    for (int w = 0; w < kSimpleWarps; ++w) {
        by[w] = part_l[w] == 0.f ? 0.f : expf(part_m[w] - top);
        sum += part_l[w] * by[w];
    }
    for (int e = threadIdx.x; e < kE; e += kSimpleWarps * 32) {
        float x = 0.f;
        for (int w = 0; w < kSimpleWarps; ++w) x += part[w][e] * by[w];
        out[e] = from_float<T>(sum == 0.f ? 0.f : x / sum);
    }
    if (lse && threadIdx.x == 0) *lse = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace topkidx
