// attend_latent.cu -- absorbed latent attention over selected slots or whole
// rows of the paged cache: one block per query head.
#include <cuda_runtime.h>

#include <cstdint>

#include "attend_internal.h"
#include "attend_simple.cuh"

namespace topkidx {
namespace {

template <typename T>
__global__ void __launch_bounds__(kSimpleWarps * 32) latent_kernel(const LatentParams p) {
    const int64_t m = blockIdx.x;
    const int h = static_cast<int>(m % p.heads), i = static_cast<int>(m / p.heads % p.queries);
    const int64_t b = m / p.heads / p.queries;
    const T* q = static_cast<const T*>(p.q) + b * p.q_row_stride + i * p.q_query_stride + h * p.q_head_stride;
    int n = p.max_len;
    if (p.seq_lens) n = min(max(p.seq_lens[b], 0), n);
    n = max(n - (p.queries - 1 - i), 0);
    const auto slot_of = [&](int j) -> int32_t {
        if (p.indices) return p.indices[b * p.indices_stride + j];
        const int64_t s = (static_cast<int64_t>(p.table[b * p.table_stride + (j >> p.log2_page)]) << p.log2_page) +
                          (j & ((1 << p.log2_page) - 1));
        return s >= 0 && s < p.num_slots ? static_cast<int32_t>(s) : -1;
    };
    const T* row = nullptr;
    simple_attend<T, kWidth, kLatent>(
        n, p.scale, [&](int d) { return to_float(q[d]); },
        [&](int j) {
            const int32_t s = slot_of(j);
            row = static_cast<const T*>(p.cache) + static_cast<int64_t>(s) * p.slot_stride;
            return s >= 0 && s < p.num_slots;
        },
        [&](int, int d) { return to_float(row[d]); }, [&](int, int d) { return to_float(row[d]); },
        static_cast<T*>(p.out) + m * kLatent, p.lse ? p.lse + m : nullptr);
}

}  // namespace

size_t latent_workspace_bytes(int32_t, int32_t, int32_t) { return 16; }

topk_status_t launch_latent(const LatentParams& p, topk_dtype_t dtype, cudaStream_t stream) {
    const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(p.batch) * p.queries * p.heads);
    if (dtype == TOPK_BF16)
        latent_kernel<__nv_bfloat16><<<blocks, kSimpleWarps * 32, 0, stream>>>(p);
    else
        latent_kernel<__half><<<blocks, kSimpleWarps * 32, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TOPK_OK : api_cuda_fail(e, "latent attention launch");
}

}  // namespace topkidx
