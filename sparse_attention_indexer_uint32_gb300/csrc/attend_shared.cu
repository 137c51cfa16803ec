// attend_shared.cu -- topk_attend_shared: latent attention for requests whose
// first positions are the same.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attend_internal.h"
#include "ptx.cuh"
#include "two_byte.cuh"

namespace topkidx {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// One (query, head) row a block; each warp takes every eighth position with a
// running maximum of its own.
template <typename T>
__global__ void __launch_bounds__(kThreads) shared_kernel(const LatentParams p) {
    __shared__ float tops[kWarps], sums[kWarps], values[kWarps][kLatent];
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int64_t row = blockIdx.x;
    const int h = static_cast<int>(row % p.heads), i = static_cast<int>(row / p.heads % p.queries),
              b = static_cast<int>(row / p.heads / p.queries);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int length = min(max(p.seq_lens[b], 0), p.max_len), limit = length - (p.queries - 1 - i);
    const int shared = min(max(*p.shared_len, 0), p.max_shared);
    const T* q = static_cast<const T*>(p.q) + b * p.q_row_stride + i * p.q_query_stride + h * p.q_head_stride;
    float m = -INFINITY, l = 0.f, o[16] = {}, x[18];
    for (int v = 0; v < 18; ++v) x[v] = static_cast<float>(q[lane + 32 * v]);
    for (int t = warp; t < limit; t += kWarps) {
        const int page = t < shared ? p.shared_pages[t >> p.log2_page] : p.table[b * p.table_stride + (t >> p.log2_page)];
        const int64_t slot = (static_cast<int64_t>(page) << p.log2_page) + (t & ((1 << p.log2_page) - 1));
        if (slot < 0 || slot >= p.num_slots) continue;
        const T* c = static_cast<const T*>(p.cache) + slot * p.slot_stride;
        float k[18], dot = 0.f;
        for (int v = 0; v < 18; ++v) k[v] = static_cast<float>(c[lane + 32 * v]);
        for (int v = 0; v < 18; ++v) dot += x[v] * k[v];
        for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(~0u, dot, d);
        const float s = dot * p.scale, top = fmaxf(m, s), by = m == -INFINITY ? 0.f : expf(m - top), w = expf(s - top);
        m = top;
        l = l * by + w;
        for (int v = 0; v < 16; ++v) o[v] = o[v] * by + w * k[v];
    }
    if (lane == 0) {
        tops[warp] = m;
        sums[warp] = l;
    }
    for (int v = 0; v < 16; ++v) values[warp][lane + 32 * v] = o[v];
    __syncthreads();
    float top = -INFINITY, total = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, tops[w]);
    for (int w = 0; w < kWarps; ++w)
        if (sums[w] > 0.f) total += sums[w] * expf(tops[w] - top);
    for (int v = threadIdx.x; v < kLatent; v += kThreads) {
        float sum = 0.f;
        for (int w = 0; w < kWarps; ++w)
            if (sums[w] > 0.f) sum += values[w][v] * expf(tops[w] - top);
        static_cast<T*>(p.out)[row * kLatent + v] = static_cast<T>(total > 0.f ? sum / total : 0.f);
    }
    if (p.lse && threadIdx.x == 0) p.lse[row] = total > 0.f ? top + logf(total) : -INFINITY;
}

}  // namespace

size_t shared_workspace_bytes(int32_t, int32_t, int32_t) { return 16; }

topk_status_t launch_shared(const LatentParams& p, topk_dtype_t dtype, const AttendDevice&, cudaStream_t stream) {
    const auto kernel = dtype == TOPK_BF16 ? shared_kernel<__nv_bfloat16> : shared_kernel<__half>;
    const int64_t rows = static_cast<int64_t>(p.batch) * p.queries * p.heads;
    const cudaError_t e = launch_early(kernel, dim3(static_cast<unsigned>(rows)), kThreads, 0, stream, p);
    return e == cudaSuccess ? TOPK_OK : api_cuda_fail(e, "shared attention launch");
}

}  // namespace topkidx
