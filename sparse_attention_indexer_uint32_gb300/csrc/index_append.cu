// index_append.cu -- topk_index_append: layer norm, rotation and paged store
// of the indexer's keys in one pass.
//
// Mathematics: y = (x - mean x) / sqrt(mean (x - mean x)^2 + eps) w + b over 128
// values in fp32 (the mean first, then the squares of what is left: no
// difference of two large sums), then the rotation of 64 of them by the angle
// of the token's position, and one rounding.  Half a warp holds a key, eight
// values (16 bytes) a lane, so a key is read once and written once: 256 + 256 +
// 256 bytes with its cosines and sines, bound by memory at large counts and by the
// call at small ones.  65536 keys take 12.0 to 12.5 us in fp16, 4.1 to 4.2 TB/s (60 to
// 62 % of the measured copy rate), and 13.3 to 13.9 in bf16, 3.7 to 3.8 TB/s: two
// dependent reads, position and angles, in each round of blocks, 4.5 rounds with
// fp16's 40 registers and 5.4 with bf16's 48.  Four keys a half warp at once took
// 15.7 us, the registers held fewer keys on an SM; 64 keys 2.9 us a call, the
// host's 2.8 of them.
#include <cuda_runtime.h>

#include <cstdint>

#include "attend_internal.h"
#include "ptx.cuh"
#include "two_byte.cuh"

namespace topkidx {
namespace {

constexpr int kThreads = 128;
constexpr int kLanes = kIndex / 8;            // lanes of a key
constexpr int kTurnLanes = kRope / 8;         // of them, those with rotary values
constexpr int kKeys = kThreads / kLanes;      // keys of a block

template <typename T>
__global__ void __launch_bounds__(kThreads) index_append_kernel(const IndexAppendParams p) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int j = threadIdx.x % kLanes, turn_lane = j - (p.rope_last ? kLanes - kTurnLanes : 0);
    const bool turns = p.cos_sin && turn_lane >= 0 && turn_lane < kTurnLanes;
    const int64_t token = static_cast<int64_t>(blockIdx.x) * kKeys + threadIdx.x / kLanes;
    int32_t slot = -1, position = 0;
    Eight<T> x = {};
    if (token < p.tokens) {
        slot = p.slots[token];
        if (p.cos_sin) position = p.positions[token];
        x = reinterpret_cast<const Eight<T>*>(static_cast<const T*>(p.rows) + token * p.row_stride)[j];
    }
    Eight<T> weight = {}, bias = {};
    if (p.weight) weight = static_cast<const Eight<T>*>(p.weight)[j];
    if (p.bias) bias = static_cast<const Eight<T>*>(p.bias)[j];
    // Interleaved, a lane's values are four pairs; else eight halves of pairs,
    // the others' halves four lanes away.
    float4 cosine[2], sine[2];
    if (slot >= p.num_slots || (p.cos_sin && (position < 0 || position >= p.num_positions))) slot = -1;
    if (turns && slot >= 0) {
        const float4* turn = reinterpret_cast<const float4*>(p.cos_sin + static_cast<int64_t>(position) * kRope);
        const int at = p.interleaved ? turn_lane : 2 * (turn_lane & 3);
        cosine[0] = turn[at];
        sine[0] = turn[kRope / 8 + at];
        if (!p.interleaved) {
            cosine[1] = turn[at + 1];
            sine[1] = turn[kRope / 8 + at + 1];
        }
    }
    float f[8];
    widen(x, f);
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
        float w[8], b[8];
        widen(weight, w);
        widen(bias, b);
#pragma unroll
        for (int v = 0; v < 8; ++v) f[v] = fmaf(f[v] * by, w[v], b[v]);
    }
    if (p.cos_sin && p.interleaved) {
        if (turns && slot >= 0) {
            const float c[4] = {cosine[0].x, cosine[0].y, cosine[0].z, cosine[0].w};
            const float s[4] = {sine[0].x, sine[0].y, sine[0].z, sine[0].w};
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
        if (turns && slot >= 0) {
            const float c[8] = {cosine[0].x, cosine[0].y, cosine[0].z, cosine[0].w,
                                cosine[1].x, cosine[1].y, cosine[1].z, cosine[1].w};
            const float s[8] = {sine[0].x, sine[0].y, sine[0].z, sine[0].w,
                                sine[1].x, sine[1].y, sine[1].z, sine[1].w};
#pragma unroll
            for (int v = 0; v < 8; ++v)
                f[v] = turn_lane < kTurnLanes / 2 ? f[v] * c[v] - other[v] * s[v] : other[v] * s[v] + f[v] * c[v];
        }
    }
    if (slot >= 0)
        reinterpret_cast<Eight<T>*>(static_cast<T*>(p.cache) + static_cast<int64_t>(slot) * p.slot_stride)[j] = narrow<T>(f);
}

}  // namespace

cudaError_t launch_index_append(const IndexAppendParams& p, topk_dtype_t dtype, cudaStream_t stream) {
    const int64_t blocks = (static_cast<int64_t>(p.tokens) + kKeys - 1) / kKeys;
    return launch_early(dtype == TOPK_BF16 ? index_append_kernel<__nv_bfloat16> : index_append_kernel<__half>,
                        dim3(static_cast<unsigned>(blocks)), kThreads, 0, stream, p);
}

}  // namespace topkidx
