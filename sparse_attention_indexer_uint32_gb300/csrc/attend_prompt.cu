// attend_prompt.cu -- expanded latent attention for prompts: one block per
// query head.
#include <cuda_runtime.h>

#include <cstdint>

#include "attend_internal.h"
#include "attend_simple.cuh"

namespace topkidx {
namespace {

template <typename T>
__global__ void __launch_bounds__(kSimpleWarps * 32) prompt_kernel(const PromptParams p) {
    const int64_t m = blockIdx.x;
    const int h = static_cast<int>(m % p.heads);
    const int64_t t = m / p.heads;
    int b = -1, q0 = 0, q1 = 0;
    for (int r = 0; r < p.batch; ++r) {
        const int lo = min(max(p.cu_q[r], 0), p.total_q), hi = min(max(p.cu_q[r + 1], lo), p.total_q);
        if (t >= lo && t < hi) {
            b = r;
            q0 = lo;
            q1 = hi;
            break;
        }
    }
    if (b < 0) return;
    const int k0 = min(max(p.cu_k[b], 0), p.total_k), k1 = min(max(p.cu_k[b + 1], k0), p.total_k);
    int n = k1 - k0;
    if (p.causal) n = max(n - (q1 - 1 - static_cast<int>(t)), 0);
    const T* q = static_cast<const T*>(p.q) + t * p.q_token_stride + h * p.q_head_stride;
    const T* kn = static_cast<const T*>(p.k_nope) + k0 * p.k_token_stride + h * p.k_head_stride;
    const T* kr = static_cast<const T*>(p.k_rope) + k0 * p.k_rope_stride;
    const T* v = static_cast<const T*>(p.v) + k0 * p.v_token_stride + h * p.v_head_stride;
    simple_attend<T, kNope + kRope, kValue>(
        n, p.scale, [&](int d) { return to_float(q[d]); }, [&](int) { return true; },
        [&](int j, int d) {
            return to_float(d < kNope ? kn[j * p.k_token_stride + d] : kr[j * p.k_rope_stride + d - kNope]);
        },
        [&](int j, int d) { return to_float(v[j * p.v_token_stride + d]); }, static_cast<T*>(p.out) + m * kValue,
        p.lse ? p.lse + m : nullptr);
}

}  // namespace

topk_status_t launch_prompt(const PromptParams& p, topk_dtype_t dtype, cudaStream_t stream) {
    const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(p.total_q) * p.heads);
    if (dtype == TOPK_BF16)
        prompt_kernel<__nv_bfloat16><<<blocks, kSimpleWarps * 32, 0, stream>>>(p);
    else
        prompt_kernel<__half><<<blocks, kSimpleWarps * 32, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TOPK_OK : api_cuda_fail(e, "prompt attention launch");
}

}  // namespace topkidx
