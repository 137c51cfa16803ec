// attend_internal.h -- launch parameters of the block-table, append, index-score
// and attention kernels, shared by the host side of the ABI (attend_api.cu).
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "topkidx.h"

namespace topkidx {

constexpr int kLatent = TOPK_LATENT_DIM;
constexpr int kRope = TOPK_ROPE_DIM;
constexpr int kWidth = kLatent + kRope;
constexpr int kNope = TOPK_NOPE_DIM;
constexpr int kValue = TOPK_VALUE_DIM;
constexpr int kIndex = TOPK_INDEX_DIM;

// The ABI's device check and CUDA-error record (topkidx_api.cu).
topk_status_t api_check_device();
topk_status_t api_cuda_fail(cudaError_t e, const char* where);

// How long a wait of a kernel may take (the tuning's wait_limit_us).  A
// sleeping probe outlasts a short limit, and polling for it cost 2 to 5 % of a
// call: up to 100 us there is none, and blocks begin as if one had given up.
struct WaitLimit {
    uint64_t ns;
    uint32_t none;
};

// The current device, as the attention launches need it.
struct AttendDevice {
    static constexpr int kMax = 64;
    int index = 0;
    int sms = 0;
    uint32_t* flags = nullptr;  // where a wait that gave up is noted
};

// Lets a kernel take `bytes` of shared memory, once per kernel and device
// (`done`; a second thread that comes in between sets the same value).
template <typename Kernel>
cudaError_t allow_shared(Kernel kernel, int bytes, std::atomic<bool>& done) {
    if (done.load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.store(true, std::memory_order_release);
    return e;
}

// Launches a kernel that may be placed before the kernel ahead of it in the
// stream has ended; it waits (griddepcontrol.wait) before its first access.
// `cluster`: blocks of a cluster, 0 for what the kernel itself says.
template <typename... Params, typename... Args>
cudaError_t launch_early_clusters(void (*kernel)(Params...), dim3 grid, int cluster, int threads, size_t shared,
                                  cudaStream_t stream, const Args&... args) {
    cudaLaunchAttribute attrs[2] = {};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
    return e == cudaSuccess ? cudaGetLastError() : e;
}
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, size_t shared, cudaStream_t stream,
                         const Args&... args) {
    return launch_early_clusters(kernel, grid, 0, threads, shared, stream, args...);
}

// Clusters of a kernel that the current device holds at once.
template <typename Kernel>
cudaError_t clusters_at_once(int* count, Kernel kernel, int threads, size_t shared, int cluster) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(cluster);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = shared;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(count, kernel, &cfg);
}

struct TablesParams {
    const int32_t* context;
    const int32_t* fresh;
    int32_t batch;
    int32_t log2_page;
    const int32_t* free_pages;
    int32_t num_free;
    int32_t* table;
    int64_t table_stride;
    int32_t width;
    int32_t max_tokens;
    int32_t* seq_lens;
    int32_t* cu_new;
    int32_t* slots;
    int32_t* positions;  // or null
    int32_t* rows;       // or null
    int32_t* status;
};
cudaError_t launch_block_tables(const TablesParams& p, cudaStream_t stream);

struct AppendParams {
    const void* rows;
    int64_t row_stride;
    int32_t tokens;
    const void* weight;  // or null
    float eps;
    const float* cos_sin;  // or null
    int32_t num_positions;
    const int32_t* positions;
    const int32_t* slots;
    void* cache;
    int64_t slot_stride;
    int32_t num_slots;
};
cudaError_t launch_cache_append(const AppendParams& p, bool interleaved, topk_dtype_t dtype, cudaStream_t stream);

struct IndexAppendParams {
    const void* rows;
    int64_t row_stride;
    int32_t tokens;
    const void* weight;  // or null
    const void* bias;    // or null
    float eps;
    const float* cos_sin;  // or null
    int32_t num_positions;
    const int32_t* positions;
    bool interleaved, rope_last;
    const int32_t* slots;
    void* cache;
    int64_t slot_stride;
    int32_t num_slots;
};
cudaError_t launch_index_append(const IndexAppendParams& p, topk_dtype_t dtype, cudaStream_t stream);

struct IndexScoresParams {
    const void* q;
    int64_t q_token_stride, q_head_stride;
    const float* weights;
    int64_t weights_stride;
    const void* cache;
    int64_t slot_stride;
    int32_t num_slots;
    const int32_t* seq_lens;
    const int32_t* table;
    int64_t table_stride;
    int32_t log2_page;
    int32_t max_len;
    const int32_t* cu_q;  // null: total_q / batch queries each
    int32_t batch, total_q, heads;
    float* scores;
    int64_t scores_stride;
    WaitLimit wait;
};
topk_status_t launch_index_scores(const IndexScoresParams& p, topk_dtype_t dtype, const AttendDevice& device, cudaStream_t stream);

// Absorbed latent attention: `batch` rows of queries x heads query heads over
// up to max_len slots each, listed in `indices` or reached through `table`.
struct LatentParams {
    const void* q;
    int64_t q_row_stride, q_query_stride, q_head_stride;
    const void* cache;
    int64_t slot_stride;
    int32_t num_slots;
    const int32_t* indices;  // null: through the page table
    int64_t indices_stride;
    const int32_t* seq_lens;  // null: every row has max_len indices
    const int32_t* table;
    int64_t table_stride;
    int32_t log2_page;
    int32_t max_len;
    int32_t batch, queries, heads;
    float scale;
    void* out;
    float* lse;  // or null
    void* workspace;
    WaitLimit wait;
    // Positions that all rows share come through a page list of their own.
    const int32_t* shared_pages;
    const int32_t* shared_len;  // null: nothing is shared
    int32_t max_shared;
};
size_t latent_workspace_bytes(int32_t batch, int32_t queries, int32_t heads);
topk_status_t launch_latent(const LatentParams& p, topk_dtype_t dtype, const AttendDevice& device, cudaStream_t stream);
size_t shared_workspace_bytes(int32_t batch, int32_t queries, int32_t heads);

struct PromptParams {
    const void* q;
    int64_t q_token_stride, q_head_stride;
    const void* k_nope;
    int64_t k_token_stride, k_head_stride;
    const void* k_rope;
    int64_t k_rope_stride;
    const void* v;
    int64_t v_token_stride, v_head_stride;
    const int32_t* cu_q;
    const int32_t* cu_k;
    int32_t batch, total_q, total_k, heads;
    float scale;
    int32_t causal;
    void* out;
    float* lse;  // or null
    WaitLimit wait;
};
topk_status_t launch_prompt(const PromptParams& p, topk_dtype_t dtype, const AttendDevice& device, cudaStream_t stream);

}  // namespace topkidx
