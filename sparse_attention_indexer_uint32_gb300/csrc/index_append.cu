// index_append.cu -- topk_index_append: layer norm, rotation and paged store
// of the indexer's keys in one pass.
//
// Mathematics: y = (x - mean x) / sqrt(mean (x - mean x)^2 + eps) w + b over 128
// values in fp32 (the mean first, then the squares of what is left: no
// difference of two large sums), then the rotation of 64 of them by the angle
// of the token's position, and one rounding.  Half a warp holds a key, eight
// values (16 bytes) a lane, so a key is read once and written once.
#include <cuda_runtime.h>

#include <cstdint>

#include "attend_internal.h"
#include "ptx.cuh"
#include "two_byte.cuh"

namespace topkidx {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = kIndex / 8;            // lanes of a key
constexpr int kTurnLanes = kRope / 8;         // of them, those with rotary values
constexpr int kKeys = kThreads / kLanes;      // keys of a block at a time

// kMany keys for each half warp, their loads all under way at once.
template <typename T, int kMany>
__global__ void __launch_bounds__(kThreads) index_append_kernel(const IndexAppendParams p) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int j = threadIdx.x % kLanes, turn_lane = j - (p.rope_last ? kLanes - kTurnLanes : 0);
    const bool turns = p.cos_sin && turn_lane >= 0 && turn_lane < kTurnLanes;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kKeys * kMany) + threadIdx.x / kLanes;

    Eight<T> x[kMany];
    int32_t slot[kMany], position[kMany];
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
        const int64_t token = first + i * kKeys;
        slot[i] = -1;
        position[i] = 0;
        if (token < p.tokens) {
            slot[i] = p.slots[token];
            if (p.cos_sin) position[i] = p.positions[token];
            x[i] = reinterpret_cast<const Eight<T>*>(static_cast<const T*>(p.rows) + token * p.row_stride)[j];
        } else {
            x[i] = Eight<T>{};
        }
    }
    float w[8], b[8];
    if (p.weight) {
        widen(static_cast<const Eight<T>*>(p.weight)[j], w);
#pragma unroll
        for (int v = 0; v < 8; ++v) b[v] = 0.f;
        if (p.bias) widen(static_cast<const Eight<T>*>(p.bias)[j], b);
    }
    // Interleaved, a lane's values are four pairs; else eight halves of pairs,
    // the others' halves four lanes away.
    float4 cosine[kMany][2], sine[kMany][2];
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
        if (slot[i] >= p.num_slots || (p.cos_sin && (position[i] < 0 || position[i] >= p.num_positions))) slot[i] = -1;
        if (turns && slot[i] >= 0) {
            const float4* turn = reinterpret_cast<const float4*>(p.cos_sin + static_cast<int64_t>(position[i]) * kRope);
            const int at = p.interleaved ? turn_lane : 2 * (turn_lane & 3);
            cosine[i][0] = turn[at];
            sine[i][0] = turn[kRope / 8 + at];
            if (!p.interleaved) {
                cosine[i][1] = turn[at + 1];
                sine[i][1] = turn[kRope / 8 + at + 1];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
        float f[8];
        widen(x[i], f);
        if (p.weight) {
            float sum = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
#pragma unroll
            for (int d = kLanes / 2; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
            const float mean = sum * (1.f / kIndex);
            float square = 0.f;
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                f[v] -= mean;
                square += f[v] * f[v];
            }
#pragma unroll
            for (int d = kLanes / 2; d; d >>= 1) square += __shfl_xor_sync(~0u, square, d);
            const float by = rsqrtf(square * (1.f / kIndex) + p.eps);
#pragma unroll
            for (int v = 0; v < 8; ++v) f[v] = fmaf(f[v] * by, w[v], b[v]);
        }
        if (p.cos_sin && p.interleaved) {
            if (turns && slot[i] >= 0) {
                const float c[4] = {cosine[i][0].x, cosine[i][0].y, cosine[i][0].z, cosine[i][0].w};
                const float s[4] = {sine[i][0].x, sine[i][0].y, sine[i][0].z, sine[i][0].w};
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float a = f[2 * v], z = f[2 * v + 1];
                    f[2 * v] = a * c[v] - z * s[v];
                    f[2 * v + 1] = a * s[v] + z * c[v];
                }
            }
        } else if (p.cos_sin) {
            float other[8];
#pragma unroll
            for (int v = 0; v < 8; ++v) other[v] = __shfl_xor_sync(~0u, f[v], kTurnLanes / 2);
            if (turns && slot[i] >= 0) {
                const float c[8] = {cosine[i][0].x, cosine[i][0].y, cosine[i][0].z, cosine[i][0].w,
                                    cosine[i][1].x, cosine[i][1].y, cosine[i][1].z, cosine[i][1].w};
                const float s[8] = {sine[i][0].x, sine[i][0].y, sine[i][0].z, sine[i][0].w,
                                    sine[i][1].x, sine[i][1].y, sine[i][1].z, sine[i][1].w};
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    f[v] = turn_lane < kTurnLanes / 2 ? f[v] * c[v] - other[v] * s[v] : other[v] * s[v] + f[v] * c[v];
            }
        }
        if (slot[i] >= 0)
            reinterpret_cast<Eight<T>*>(static_cast<T*>(p.cache) + static_cast<int64_t>(slot[i]) * p.slot_stride)[j] = narrow<T>(f);
    }
}

template <typename T>
cudaError_t launch(const IndexAppendParams& p, int sms, cudaStream_t stream) {
    // Few keys: one for each half warp, over as many SMs as there are.
    const int many = p.tokens > kKeys * sms ? 4 : 1;
    const int64_t blocks = (static_cast<int64_t>(p.tokens) + kKeys * many - 1) / (kKeys * many);
    return launch_early(many == 4 ? index_append_kernel<T, 4> : index_append_kernel<T, 1>, dim3(static_cast<unsigned>(blocks)),
                        kThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_index_append(const IndexAppendParams& p, topk_dtype_t dtype, const AttendDevice& device, cudaStream_t stream) {
    return dtype == TOPK_BF16 ? launch<__nv_bfloat16>(p, device.sms, stream) : launch<__half>(p, device.sms, stream);
}

}  // namespace topkidx
