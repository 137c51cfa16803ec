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
constexpr int kTokens = 2;  // of a warp, so that more loads are in flight

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
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kTokens;
    // Everything that does not hang on another load is asked for at once, that
    // of a row without a slot too.
    Eight<T> a[kTokens], b[kTokens], r0[kTokens], r1[kTokens];
    int32_t slot[kTokens], position[kTokens];
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
        slot[k] = -1;
        position[k] = 0;
        if (first + k >= p.tokens) continue;
        slot[k] = p.slots[first + k];
        if (p.cos_sin) position[k] = p.positions[first + k];
        const Eight<T>* in = reinterpret_cast<const Eight<T>*>(static_cast<const T*>(p.rows) + (first + k) * p.row_stride);
        a[k] = in[lane];
        b[k] = in[lane + 32];
        // Lanes 0..7 hold eight neighbouring rotary values each, or lanes 0..3
        // eight of each half.
        if (lane < 8) r0[k] = in[kLatent / 8 + lane];
        if (!kInterleaved && lane < 4) r1[k] = in[kLatent / 8 + 4 + lane];
    }
    float4 c0[kTokens], s0[kTokens], c1[kTokens], s1[kTokens];
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
        if (slot[k] >= p.num_slots || (p.cos_sin && (position[k] < 0 || position[k] >= p.num_positions))) slot[k] = -1;
        if (slot[k] < 0 || !p.cos_sin || lane >= (kInterleaved ? 8 : 4)) continue;
        const float4* turn = reinterpret_cast<const float4*>(p.cos_sin + static_cast<int64_t>(position[k]) * kRope);
        const int at = kInterleaved ? lane : 2 * lane;
        c0[k] = turn[at];
        s0[k] = turn[kRope / 8 + at];
        if (!kInterleaved) {
            c1[k] = turn[at + 1];
            s1[k] = turn[kRope / 8 + at + 1];
        }
    }
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
        if (slot[k] < 0) continue;  // the whole warp
        Eight<T>* out = reinterpret_cast<Eight<T>*>(static_cast<T*>(p.cache) + static_cast<int64_t>(slot[k]) * p.slot_stride);
        if (p.weight) {
            float x[16], w[16];
            widen(a[k], x);
            widen(b[k], x + 8);
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
            out[lane] = a[k];
            out[lane + 32] = b[k];
        }
        if (lane < 8) {
            if (!p.cos_sin) {
                out[kLatent / 8 + lane] = r0[k];
            } else if (kInterleaved) {
                float x[8], y[8];
                widen(r0[k], x);
                const float cs[4] = {c0[k].x, c0[k].y, c0[k].z, c0[k].w}, sn[4] = {s0[k].x, s0[k].y, s0[k].z, s0[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[2 * i] = x[2 * i] * cs[i] - x[2 * i + 1] * sn[i];
                    y[2 * i + 1] = x[2 * i] * sn[i] + x[2 * i + 1] * cs[i];
                }
                out[kLatent / 8 + lane] = narrow<T>(y);
            } else if (lane < 4) {
                float x[8], z[8], y[8], u[8];
                widen(r0[k], x);
                widen(r1[k], z);
                const float cs[8] = {c0[k].x, c0[k].y, c0[k].z, c0[k].w, c1[k].x, c1[k].y, c1[k].z, c1[k].w};
                const float sn[8] = {s0[k].x, s0[k].y, s0[k].z, s0[k].w, s1[k].x, s1[k].y, s1[k].z, s1[k].w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[i] = x[i] * cs[i] - z[i] * sn[i];
                    u[i] = x[i] * sn[i] + z[i] * cs[i];
                }
                out[kLatent / 8 + lane] = narrow<T>(y);
                out[kLatent / 8 + 4 + lane] = narrow<T>(u);
            }
        }
        __syncwarp();
    }
}

template <typename T>
cudaError_t launch(const AppendParams& p, bool interleaved, cudaStream_t stream) {
    constexpr int kBlockTokens = kThreads / 32 * kTokens;
    const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(p.tokens) + kBlockTokens - 1) / kBlockTokens);
    return launch_early(interleaved ? cache_append_kernel<T, true> : cache_append_kernel<T, false>, dim3(blocks), kThreads,
                        0, stream, p);
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams& p, bool interleaved, topk_dtype_t dtype, cudaStream_t stream) {
    return dtype == TOPK_BF16 ? launch<__nv_bfloat16>(p, interleaved, stream) : launch<__half>(p, interleaved, stream);
}

}  // namespace topkidx
