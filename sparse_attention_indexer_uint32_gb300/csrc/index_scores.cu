// index_scores.cu -- topk_index_scores: weighted scores of the indexer's heads
// over its paged keys.
//
// Mathematics: I[i][t] = sum_h w[i][h] max(q[i][h].k[t], 0) over 128 values a
// head.  Products of two-byte values are exact in fp32; all sums are fp32.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attend_internal.h"
#include "ptx.cuh"
#include "two_byte.cuh"

namespace topkidx {
namespace {

constexpr int kThreads = 256;

// One query a block, one key a half warp at a time.
template <typename T>
__global__ void __launch_bounds__(kThreads) index_scores_kernel(const IndexScoresParams p) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int i = blockIdx.x;
    int b = -1, last = 0;
    if (p.cu_q) {
        for (int r = 0; r < p.batch; ++r)
            if (p.cu_q[r] <= i && i < p.cu_q[r + 1]) {
                b = r;
                last = min(p.cu_q[r + 1], p.total_q) - 1;
                break;
            }
    } else {
        const int n = p.total_q / p.batch;
        b = i / n;
        last = b * n + n - 1;
    }
    if (b < 0) return;
    const int limit = min(max(p.seq_lens[b], 0), p.max_len) - (last - i);
    const int j = threadIdx.x & 15;
    const T* q = static_cast<const T*>(p.q) + i * p.q_token_stride;
    for (int t0 = static_cast<int>(blockIdx.y) * (kThreads / 16); t0 < limit; t0 += static_cast<int>(gridDim.y) * (kThreads / 16)) {
        const int t = t0 + threadIdx.x / 16;
        float k[8] = {}, total = 0.f;
        bool seen = false;
        if (t < limit) {
            const int64_t slot = (static_cast<int64_t>(p.table[b * p.table_stride + (t >> p.log2_page)]) << p.log2_page) + (t & ((1 << p.log2_page) - 1));
            seen = slot >= 0 && slot < p.num_slots;
            if (seen) widen(reinterpret_cast<const Eight<T>*>(static_cast<const T*>(p.cache) + slot * p.slot_stride)[j], k);
        }
        for (int h = 0; h < p.heads; ++h) {
            float x[8], dot = 0.f;
            widen(reinterpret_cast<const Eight<T>*>(q + h * p.q_head_stride)[j], x);
#pragma unroll
            for (int v = 0; v < 8; ++v) dot += x[v] * k[v];
#pragma unroll
            for (int d = 8; d; d >>= 1) dot += __shfl_xor_sync(~0u, dot, d);
            total += p.weights[i * p.weights_stride + h] * ptx::fmax_nan(dot, 0.f);
        }
        if (t < limit && j == 0) p.scores[i * p.scores_stride + t] = seen ? total : -INFINITY;
    }
}

}  // namespace

topk_status_t launch_index_scores(const IndexScoresParams& p, topk_dtype_t dtype, const AttendDevice&, cudaStream_t stream) {
    const auto kernel = dtype == TOPK_BF16 ? index_scores_kernel<__nv_bfloat16> : index_scores_kernel<__half>;
    const cudaError_t e = launch_early(kernel, dim3(p.total_q, 32), kThreads, 0, stream, p);
    return e == cudaSuccess ? TOPK_OK : api_cuda_fail(e, "index scores launch");
}

}  // namespace topkidx
