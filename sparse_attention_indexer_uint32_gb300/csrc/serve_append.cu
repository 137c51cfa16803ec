// serve_append.cu -- topk_cache_append: norm, rotation and paged store of
// latent rows in one pass.
//
// Mathematics: c' = c rsqrt(mean(c^2) + eps) w in fp32; the rotation turns
// pair (a, b) by the angle of its position.  One warp holds one row in
// registers (16 latent values a lane in two 16-byte loads; the 64 rotary
// values in its first 8 or 4 lanes), so the row is read once and written once:
// 1152 + 256 + 1152 bytes a token, bound by memory at large counts and by the
// launch at small ones.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attend_internal.h"
#include "ptx.cuh"

namespace topkidx {
namespace {

constexpr int kThreads = 256;

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

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const AppendParams p) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t token = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (token >= p.tokens) return;
    const int32_t slot = p.slots[token];
    if (slot < 0 || slot >= p.num_slots) return;
    int32_t position = 0;
    if (p.cos_sin) {
        position = p.positions[token];
        if (position < 0 || position >= p.num_positions) return;
    }
    const Eight<T>* in = reinterpret_cast<const Eight<T>*>(static_cast<const T*>(p.rows) + token * p.row_stride);
    Eight<T>* out = reinterpret_cast<Eight<T>*>(static_cast<T*>(p.cache) + static_cast<int64_t>(slot) * p.slot_stride);
    const Eight<T> a = in[lane], b = in[lane + 32];
    Eight<T> r0, r1;
    // Lanes 0..7 hold eight neighbouring rotary values each, or lanes 0..3
    // eight of each half.
    if (lane < 8) r0 = in[kLatent / 8 + lane];
    if (!kInterleaved && lane < 4) r1 = in[kLatent / 8 + 4 + lane];
    if (p.weight) {
        float x[16], w[16];
        widen(a, x);
        widen(b, x + 8);
        float square = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) square += x[i] * x[i];
#pragma unroll
        for (int d = 16; d; d >>= 1) square += __shfl_xor_sync(~0u, square, d);
        const float by = rsqrtf(square * (1.f / kLatent) + p.eps);
        const Eight<T>* weight = static_cast<const Eight<T>*>(p.weight);
        widen(weight[lane], w);
        widen(weight[lane + 32], w + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] * by * w[i];
        out[lane] = narrow<T>(x);
        out[lane + 32] = narrow<T>(x + 8);
    } else {
        out[lane] = a;
        out[lane + 32] = b;
    }
    if (lane >= 8) return;
    if (!p.cos_sin) {
        out[kLatent / 8 + lane] = r0;
        return;
    }
    const float* turn = p.cos_sin + static_cast<int64_t>(position) * kRope;
    float x[8], y[8];
    widen(r0, x);
    if (kInterleaved) {
        const float4 c = reinterpret_cast<const float4*>(turn)[lane];
        const float4 s = reinterpret_cast<const float4*>(turn + kRope / 2)[lane];
        const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = x[2 * i] * cs[i] - x[2 * i + 1] * sn[i];
            y[2 * i + 1] = x[2 * i] * sn[i] + x[2 * i + 1] * cs[i];
        }
        out[kLatent / 8 + lane] = narrow<T>(y);
    } else if (lane < 4) {
        float z[8], u[8];
        widen(r1, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = turn[8 * lane + i], s = turn[kRope / 2 + 8 * lane + i];
            y[i] = x[i] * c - z[i] * s;
            u[i] = x[i] * s + z[i] * c;
        }
        out[kLatent / 8 + lane] = narrow<T>(y);
        out[kLatent / 8 + 4 + lane] = narrow<T>(u);
    }
}

template <typename T>
cudaError_t launch(const AppendParams& p, bool interleaved, cudaStream_t stream) {
    const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(p.tokens) + kThreads / 32 - 1) / (kThreads / 32));
    return launch_early(interleaved ? cache_append_kernel<T, true> : cache_append_kernel<T, false>, dim3(blocks), kThreads,
                        0, stream, p);
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams& p, bool interleaved, topk_dtype_t dtype, cudaStream_t stream) {
    return dtype == TOPK_BF16 ? launch<__nv_bfloat16>(p, interleaved, stream) : launch<__half>(p, interleaved, stream);
}

}  // namespace topkidx
