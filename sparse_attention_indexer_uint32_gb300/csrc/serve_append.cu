// serve_append.cu -- topk_cache_append: norm, rotation and paged store of
// latent rows in one pass.
//
// Mathematics: c' = c rsqrt(mean(c^2) + eps) w in fp32; the rotation turns
// pair (a, b) by the angle of its position.  A warp holds a row in registers
// (16 latent values a lane in two 16-byte loads, one rotary pair a lane), so the
// row is read once and written once: 1152 + 256 + 1152 bytes a token, bound by
// memory at large counts and by the launch at small ones.  Each warp walks
// several rows with the weight kept, the row after the next and the next row's
// cosines under way: 65536 rows take 31.6 us, 5.3 TB/s or 79 % of the measured
// copy rate (a warp for one row or two took 43 us, the weight's second reading
// filled the L1 path); 64 rows 7.9 us a call, most of it the host's.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attend_internal.h"
#include "ptx.cuh"

namespace topkidx {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kResident = 152 * 3;  // blocks that the GPU holds at once

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

// One row on its way; a slot below 0 is not written.
template <typename T, bool kInterleaved>
struct Row {
    Eight<T> a, b;
    typename Pair<T>::two pair;  // rotary values 2 lane, 2 lane + 1, or lane, lane + 32
    int32_t slot, position;
    float cosine, sine;

    __device__ __forceinline__ void load(const AppendParams& p, int64_t token, int lane) {
        slot = -1;
        if (token >= p.tokens) return;
        slot = p.slots[token];
        if (p.cos_sin) position = p.positions[token];
        const T* from = static_cast<const T*>(p.rows) + token * p.row_stride;
        const Eight<T>* in = reinterpret_cast<const Eight<T>*>(from);
        a = in[lane];
        b = in[lane + 32];
        if (kInterleaved) {
            pair = reinterpret_cast<const typename Pair<T>::two*>(from + kLatent)[lane];
        } else {
            pair.x = from[kLatent + lane];
            pair.y = from[kLatent + kRope / 2 + lane];
        }
    }
    __device__ __forceinline__ void load_turn(const AppendParams& p, int lane) {
        if (slot >= p.num_slots) slot = -1;
        if (slot < 0 || !p.cos_sin) return;
        if (position < 0 || position >= p.num_positions) {
            slot = -1;
            return;
        }
        const float* turn = p.cos_sin + static_cast<int64_t>(position) * kRope;
        cosine = turn[lane];
        sine = turn[kRope / 2 + lane];
    }
    __device__ __forceinline__ void store(const AppendParams& p, const float* w, int lane) const {
        if (slot < 0) return;  // the whole warp
        T* to = static_cast<T*>(p.cache) + static_cast<int64_t>(slot) * p.slot_stride;
        Eight<T>* out = reinterpret_cast<Eight<T>*>(to);
        if (p.weight) {
            float x[16];
            widen(a, x);
            widen(b, x + 8);
            float square = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) square += x[i] * x[i];
#pragma unroll
            for (int d = 16; d; d >>= 1) square += __shfl_xor_sync(~0u, square, d);
            const float by = rsqrtf(square * (1.f / kLatent) + p.eps);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = x[i] * by * w[i];
            out[lane] = narrow<T>(x);
            out[lane + 32] = narrow<T>(x + 8);
        } else {
            out[lane] = a;
            out[lane + 32] = b;
        }
        typename Pair<T>::two y = pair;
        if (p.cos_sin) {
            const float2 x = Pair<T>::wide(pair);
            y = Pair<T>::narrow(make_float2(x.x * cosine - x.y * sine, x.x * sine + x.y * cosine));
        }
        if (kInterleaved) {
            reinterpret_cast<typename Pair<T>::two*>(to + kLatent)[lane] = y;
        } else {
            to[kLatent + lane] = y.x;
            to[kLatent + kRope / 2 + lane] = y.y;
        }
    }
};

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const AppendParams p) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    int64_t token = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    Row<T, kInterleaved> now, next, later;
    now.load(p, token, lane);
    next.load(p, token + step, lane);
    float w[16];
    if (p.weight) {
        const Eight<T>* weight = static_cast<const Eight<T>*>(p.weight);
        widen(weight[lane], w);
        widen(weight[lane + 32], w + 8);
    }
    now.load_turn(p, lane);
    for (; token < p.tokens; token += step) {
        later.load(p, token + 2 * step, lane);
        next.load_turn(p, lane);
        now.store(p, w, lane);
        now = next;
        next = later;
    }
}

template <typename T>
cudaError_t launch(const AppendParams& p, bool interleaved, cudaStream_t stream) {
    const int64_t needed = (static_cast<int64_t>(p.tokens) + kThreads / 32 - 1) / (kThreads / 32);
    const unsigned blocks = static_cast<unsigned>(needed < kResident ? needed : kResident);
    return launch_early(interleaved ? cache_append_kernel<T, true> : cache_append_kernel<T, false>, dim3(blocks), kThreads,
                        0, stream, p);
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams& p, bool interleaved, topk_dtype_t dtype, cudaStream_t stream) {
    return dtype == TOPK_BF16 ? launch<__nv_bfloat16>(p, interleaved, stream) : launch<__half>(p, interleaved, stream);
}

}  // namespace topkidx
