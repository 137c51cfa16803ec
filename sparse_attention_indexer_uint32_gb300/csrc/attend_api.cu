// attend_api.cu -- host side of the block-table, append, index-score and
// attention entry points of include/topkidx.h: argument checks before any launch.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "attend_internal.h"
#include "topk_internal.h"
#include "topkidx.h"

using namespace topkidx;

namespace {

bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
bool page_ok(int32_t n) { return n >= 1 && n <= (1 << 30) && (n & (n - 1)) == 0; }
bool dtype_ok(topk_dtype_t t) { return t == TOPK_BF16 || t == TOPK_FP16; }

int log2_of(int32_t n) {
    int r = 0;
    while ((int64_t{1} << r) < n) ++r;
    return r;
}

// Rows of two-byte values: 16-byte aligned base and strides.
bool row_stride_ok(int64_t stride, int64_t least) { return stride >= least && stride <= (int64_t{1} << 38); }

// The rows of a tensor that a product reads: far enough apart not to overlap,
// unless there is only one.
bool token_stride_ok(int64_t stride, int64_t least, int64_t count) {
    return row_stride_ok(stride, count > 1 ? least : 0);
}

constexpr int64_t kMaxQueryHeads = int64_t{1} << 30;

// int32 values at an address: `rows` rows of n, `stride` apart (4-byte aligned).
struct Span {
    const int32_t* at;
    int64_t n;
    int64_t rows = 1, stride = 0;
};

// Whether a row of values and rows of values have one in common: the first of
// the rows that ends behind the start of `a` begins before its end.
bool overlap(const Span& a, const Span& b) {
    if (!a.at || !b.at || a.n <= 0 || b.n <= 0) return false;
    const auto address = [](const Span& s) { return static_cast<int64_t>(reinterpret_cast<uintptr_t>(s.at) / 4); };
    const int64_t from = address(a) - address(b);
    const int64_t past = from - b.n;  // rows that begin up to here end before `a`
    const int64_t row = past < 0 ? 0 : b.rows > 1 ? past / b.stride + 1 : 1;
    return row < b.rows && row * b.stride < from + a.n;
}

WaitLimit wait_limit() {
    topk_tuning_t t;
    (void)topk_get_tuning(&t);
    const uint64_t ns = t.wait_limit_us > 0 ? 1000ull * static_cast<uint64_t>(t.wait_limit_us) : kDefaultWaitLimitNs;
    return {ns, ns <= 100000ull ? 1u : 0u};
}

// The word in which the attention kernels note a wait that gave up, one per GPU.
__device__ uint32_t g_attend_flags;

// The current device, looked up once.
topk_status_t attend_device(AttendDevice* out) {
    static AttendDevice known[AttendDevice::kMax];
    static std::atomic<bool> looked_up[AttendDevice::kMax];
    static std::mutex mutex;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return api_cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= AttendDevice::kMax) return api_cuda_fail(cudaErrorInvalidDevice, "attention device");
    if (!looked_up[dev].load(std::memory_order_acquire)) {
        const topk_status_t st = api_check_device();
        if (st != TOPK_OK) return st;
        std::lock_guard<std::mutex> lock(mutex);
        AttendDevice d;
        d.index = dev;
        void* flags = nullptr;
        e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaGetSymbolAddress(&flags, g_attend_flags);
        if (e != cudaSuccess) return api_cuda_fail(e, "attention device");
        d.flags = static_cast<uint32_t*>(flags);
        known[dev] = d;
        looked_up[dev].store(true, std::memory_order_release);
    }
    *out = known[dev];
    return TOPK_OK;
}

}  // namespace

extern "C" {

topk_status_t topk_block_tables(const int32_t* context_lens, const int32_t* new_lens, int32_t batch,
                                int32_t page_size, const int32_t* free_pages, int32_t num_free,
                                int32_t* page_table, int64_t page_table_stride, int32_t pages_per_row,
                                int32_t max_tokens, int32_t* seq_lens, int32_t* cu_new, int32_t* slots,
                                int32_t* positions_or_null, int32_t* rows_or_null, int32_t* status,
                                topk_stream_t stream) {
    if (!context_lens || !new_lens || !page_table || !seq_lens || !cu_new || !status) return TOPK_EINVAL;
    if (batch < 1 || !page_ok(page_size) || num_free < 0 || max_tokens < 0) return TOPK_EINVAL;
    if ((num_free > 0 && !free_pages) || (max_tokens > 0 && !slots)) return TOPK_EINVAL;
    if (pages_per_row < 1 || page_table_stride < pages_per_row) return TOPK_EINVAL;
    if (static_cast<int64_t>(batch) * pages_per_row > INT32_MAX) return TOPK_EINVAL;
    if (misaligned(context_lens, 4) || misaligned(new_lens, 4) || misaligned(free_pages, 4) ||
        misaligned(page_table, 4) || misaligned(seq_lens, 4) || misaligned(cu_new, 4) || misaligned(slots, 4) ||
        misaligned(positions_or_null, 4) || misaligned(rows_or_null, 4) || misaligned(status, 4))
        return TOPK_EALIGN;
    // Lengths, pages and the list are read again after outputs are written, by
    // every block: an output in their place would change them under way.
    const Span inputs[] = {{context_lens, batch}, {new_lens, batch}, {free_pages, num_free}};
    const Span table = {page_table, pages_per_row, batch, page_table_stride};
    const Span outputs[] = {{seq_lens, batch},           {cu_new, int64_t{batch} + 1}, {slots, max_tokens},
                            {positions_or_null, max_tokens}, {rows_or_null, max_tokens},   {status, 2}};
    for (const Span& in : inputs)
        if (overlap(in, table)) return TOPK_EINVAL;
    for (const Span& out : outputs) {
        if (overlap(out, table)) return TOPK_EINVAL;
        for (const Span& in : inputs)
            if (overlap(out, in)) return TOPK_EINVAL;
    }
    const topk_status_t dev = api_check_device();
    if (dev != TOPK_OK) return dev;
    TablesParams p = {context_lens, new_lens,   batch,  log2_of(page_size), free_pages, num_free,
                      page_table,   page_table_stride, pages_per_row, max_tokens, seq_lens, cu_new,
                      slots,        positions_or_null, rows_or_null, status};
    const cudaError_t e = launch_block_tables(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TOPK_OK : api_cuda_fail(e, "block table launch");
}

topk_status_t topk_cache_append(const void* rows, int64_t row_stride, int32_t tokens, const void* norm_weight_or_null,
                                float eps, const float* cos_sin_or_null, int32_t num_positions,
                                const int32_t* positions_or_null, int32_t interleaved, const int32_t* slots,
                                void* cache, int64_t slot_stride, int32_t num_slots, topk_dtype_t dtype,
                                topk_stream_t stream) {
    if (tokens < 0 || num_slots < 1 || !cache || !dtype_ok(dtype)) return TOPK_EINVAL;
    if (tokens > 0 && (!rows || !slots)) return TOPK_EINVAL;
    if (!row_stride_ok(row_stride, kWidth) || !row_stride_ok(slot_stride, kWidth)) return TOPK_EINVAL;
    if (norm_weight_or_null && !(eps >= 0.f && std::isfinite(eps))) return TOPK_EINVAL;
    if (cos_sin_or_null && (num_positions < 1 || (tokens > 0 && !positions_or_null))) return TOPK_EINVAL;
    if (misaligned(rows, 16) || misaligned(cache, 16) || row_stride % 8 || slot_stride % 8 ||
        misaligned(norm_weight_or_null, 16) || misaligned(cos_sin_or_null, 16) || misaligned(positions_or_null, 4) ||
        misaligned(slots, 4))
        return TOPK_EALIGN;
    const topk_status_t dev = api_check_device();
    if (dev != TOPK_OK) return dev;
    if (tokens == 0) return TOPK_OK;
    AppendParams p = {rows,          row_stride,        tokens, norm_weight_or_null, eps,         cos_sin_or_null,
                      num_positions, positions_or_null, slots,  cache,               slot_stride, num_slots};
    const cudaError_t e = launch_cache_append(p, interleaved != 0, dtype, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TOPK_OK : api_cuda_fail(e, "cache append launch");
}

topk_status_t topk_index_append(const void* rows, int64_t row_stride, int32_t tokens, const void* norm_weight_or_null,
                                const void* norm_bias_or_null, float eps, const float* cos_sin_or_null,
                                int32_t num_positions, const int32_t* positions_or_null, int32_t interleaved,
                                int32_t rope_last, const int32_t* slots, void* cache, int64_t slot_stride,
                                int32_t num_slots, topk_dtype_t dtype, topk_stream_t stream) {
    if (tokens < 0 || num_slots < 1 || !cache || !dtype_ok(dtype)) return TOPK_EINVAL;
    if (tokens > 0 && (!rows || !slots)) return TOPK_EINVAL;
    if (!row_stride_ok(row_stride, kIndex) || !row_stride_ok(slot_stride, kIndex)) return TOPK_EINVAL;
    if (norm_weight_or_null ? !(eps >= 0.f && std::isfinite(eps)) : norm_bias_or_null != nullptr) return TOPK_EINVAL;
    if (cos_sin_or_null && (num_positions < 1 || (tokens > 0 && !positions_or_null))) return TOPK_EINVAL;
    if (misaligned(rows, 16) || misaligned(cache, 16) || row_stride % 8 || slot_stride % 8 ||
        misaligned(norm_weight_or_null, 16) || misaligned(norm_bias_or_null, 16) || misaligned(cos_sin_or_null, 16) ||
        misaligned(positions_or_null, 4) || misaligned(slots, 4))
        return TOPK_EALIGN;
    const topk_status_t st = api_check_device();
    if (st != TOPK_OK || tokens == 0) return st;
    IndexAppendParams p = {rows,          row_stride,        tokens, norm_weight_or_null, norm_bias_or_null, eps, cos_sin_or_null,
                           num_positions, positions_or_null, interleaved != 0, rope_last != 0, slots, cache, slot_stride, num_slots};
    const cudaError_t e = launch_index_append(p, dtype, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TOPK_OK : api_cuda_fail(e, "index append launch");
}

topk_status_t topk_index_scores(const void* q, int64_t q_token_stride, int64_t q_head_stride, const float* weights,
                                int64_t weights_stride, const void* cache, int64_t slot_stride, int32_t num_slots,
                                const int32_t* seq_lens, const int32_t* page_table, int64_t page_table_stride,
                                int32_t page_size, int32_t max_seq_len, const int32_t* cu_q_or_null, int32_t batch,
                                int32_t total_q, int32_t heads, topk_dtype_t dtype, float* scores, int64_t scores_stride,
                                topk_stream_t stream) {
    if (batch < 1 || total_q < 0 || heads < 1 || heads > TOPK_INDEX_MAX_HEADS || !dtype_ok(dtype) || num_slots < 1) return TOPK_EINVAL;
    if (!cache || !seq_lens || !page_table || !page_ok(page_size) || max_seq_len < 0) return TOPK_EINVAL;
    if (total_q > 0 && (!q || !weights || !scores)) return TOPK_EINVAL;
    if (!cu_q_or_null && total_q % batch != 0) return TOPK_EINVAL;
    if ((static_cast<int64_t>(total_q) + batch) * ((static_cast<int64_t>(max_seq_len) + 127) / 128) > INT32_MAX) return TOPK_EINVAL;
    if (page_table_stride < (static_cast<int64_t>(max_seq_len) + page_size - 1) / page_size || page_table_stride < 1)
        return TOPK_EINVAL;
    if (!token_stride_ok(q_token_stride, kIndex, total_q) || !token_stride_ok(q_head_stride, kIndex, heads) ||
        !row_stride_ok(slot_stride, kIndex) || !row_stride_ok(weights_stride, total_q > 1 ? heads : 0) ||
        !row_stride_ok(scores_stride, total_q > 1 ? max_seq_len : 0))
        return TOPK_EINVAL;
    if (misaligned(q, 16) || misaligned(cache, 16) || misaligned(weights, 4) || misaligned(seq_lens, 4) ||
        misaligned(page_table, 4) || misaligned(cu_q_or_null, 4) || misaligned(scores, 4) || q_token_stride % 8 ||
        q_head_stride % 8 || slot_stride % 8)
        return TOPK_EALIGN;
    AttendDevice device;
    const topk_status_t st = attend_device(&device);
    if (st != TOPK_OK || total_q == 0 || max_seq_len == 0) return st;
    IndexScoresParams p = {q,           q_token_stride, q_head_stride, weights,       weights_stride,
                           cache,       slot_stride,    num_slots,     seq_lens,      page_table,
                           page_table_stride, log2_of(page_size), max_seq_len, cu_q_or_null, batch,
                           total_q,     heads,          scores,        scores_stride, wait_limit()};
    return launch_index_scores(p, dtype, device, reinterpret_cast<cudaStream_t>(stream));
}

size_t topk_attend_workspace_bytes(int32_t batch, int32_t queries, int32_t heads) {
    if (batch < 1 || queries < 1 || heads < 1) return 0;
    if (static_cast<int64_t>(queries) * heads > kMaxQueryHeads / batch) return 0;
    return latent_workspace_bytes(batch, queries, heads);
}

namespace {

// What the cache attentions check: the query rows, the cache, the outputs.
topk_status_t check_latent(const LatentParams& p, topk_dtype_t dtype, size_t need, size_t workspace_bytes) {
    if (!p.q || !p.cache || !p.out || !p.workspace || !dtype_ok(dtype)) return TOPK_EINVAL;
    if (need == 0 || p.num_slots < 1 || std::isnan(p.scale)) return TOPK_EINVAL;
    if (!row_stride_ok(p.slot_stride, kWidth)) return TOPK_EINVAL;
    if (!token_stride_ok(p.q_row_stride, kWidth, p.batch) || !token_stride_ok(p.q_query_stride, kWidth, p.queries) ||
        !token_stride_ok(p.q_head_stride, kWidth, p.heads))
        return TOPK_EINVAL;
    if (workspace_bytes < need) return TOPK_ENOSPACE;
    if (misaligned(p.q, 16) || misaligned(p.cache, 16) || misaligned(p.out, 32) || misaligned(p.workspace, 16) ||
        misaligned(p.lse, 4) || misaligned(p.indices, 4) || misaligned(p.seq_lens, 4) || misaligned(p.table, 4) ||
        p.q_row_stride % 8 || p.q_query_stride % 8 || p.q_head_stride % 8 || p.slot_stride % 8)
        return TOPK_EALIGN;
    return TOPK_OK;
}

topk_status_t run_latent(LatentParams& p, topk_dtype_t dtype, cudaStream_t stream) {
    AttendDevice device;
    const topk_status_t st = attend_device(&device);
    p.wait = wait_limit();
    return st == TOPK_OK ? launch_latent(p, dtype, device, stream) : st;
}

}  // namespace

topk_status_t topk_attend_selected(const void* q, int64_t q_row_stride, int64_t q_head_stride, const void* cache,
                                   int64_t slot_stride, int32_t num_slots, const int32_t* indices,
                                   int64_t indices_stride, const int32_t* seq_lens_or_null, int32_t rows,
                                   int32_t heads, int32_t k, float scale, topk_dtype_t dtype, void* out,
                                   float* lse_or_null, void* workspace, size_t workspace_bytes,
                                   topk_stream_t stream) {
    if (!indices || k < 1 || indices_stride < k) return TOPK_EINVAL;
    LatentParams p = {};
    p.q = q;
    p.q_row_stride = q_row_stride;
    p.q_head_stride = q_head_stride;
    p.cache = cache;
    p.slot_stride = slot_stride;
    p.num_slots = num_slots;
    p.indices = indices;
    p.indices_stride = indices_stride;
    p.seq_lens = seq_lens_or_null;
    p.max_len = k;
    p.batch = rows;
    p.queries = 1;
    p.heads = heads;
    p.scale = scale;
    p.out = out;
    p.lse = lse_or_null;
    p.workspace = workspace;
    const topk_status_t st = check_latent(p, dtype, topk_attend_workspace_bytes(p.batch, p.queries, p.heads), workspace_bytes);
    return st == TOPK_OK ? run_latent(p, dtype, reinterpret_cast<cudaStream_t>(stream)) : st;
}

topk_status_t topk_attend_paged(const void* q, int64_t q_row_stride, int64_t q_query_stride, int64_t q_head_stride,
                                const void* cache, int64_t slot_stride, int32_t num_slots, const int32_t* seq_lens,
                                const int32_t* page_table, int64_t page_table_stride, int32_t page_size,
                                int32_t max_seq_len, int32_t batch, int32_t queries, int32_t heads, float scale,
                                topk_dtype_t dtype, void* out, float* lse_or_null, void* workspace,
                                size_t workspace_bytes, topk_stream_t stream) {
    if (!seq_lens || !page_table || !page_ok(page_size) || max_seq_len < 0) return TOPK_EINVAL;
    if (page_table_stride < (static_cast<int64_t>(max_seq_len) + page_size - 1) / page_size || page_table_stride < 1)
        return TOPK_EINVAL;
    LatentParams p = {};
    p.q = q;
    p.q_row_stride = q_row_stride;
    p.q_query_stride = q_query_stride;
    p.q_head_stride = q_head_stride;
    p.cache = cache;
    p.slot_stride = slot_stride;
    p.num_slots = num_slots;
    p.seq_lens = seq_lens;
    p.table = page_table;
    p.table_stride = page_table_stride;
    p.log2_page = log2_of(page_size);
    p.max_len = max_seq_len;
    p.batch = batch;
    p.queries = queries;
    p.heads = heads;
    p.scale = scale;
    p.out = out;
    p.lse = lse_or_null;
    p.workspace = workspace;
    const topk_status_t st = check_latent(p, dtype, topk_attend_workspace_bytes(p.batch, p.queries, p.heads), workspace_bytes);
    return st == TOPK_OK ? run_latent(p, dtype, reinterpret_cast<cudaStream_t>(stream)) : st;
}

size_t topk_attend_shared_workspace_bytes(int32_t batch, int32_t queries, int32_t heads) {
    if (topk_attend_workspace_bytes(batch, queries, heads) == 0) return 0;
    return shared_workspace_bytes(batch, queries, heads);
}

topk_status_t topk_attend_shared(const void* q, int64_t q_row_stride, int64_t q_query_stride, int64_t q_head_stride,
                                 const void* cache, int64_t slot_stride, int32_t num_slots, const int32_t* seq_lens,
                                 const int32_t* page_table, int64_t page_table_stride, const int32_t* shared_pages,
                                 int32_t num_shared_pages, const int32_t* shared_len, int32_t page_size,
                                 int32_t max_seq_len, int32_t batch, int32_t queries, int32_t heads, float scale,
                                 topk_dtype_t dtype, void* out, float* lse_or_null, void* workspace,
                                 size_t workspace_bytes, topk_stream_t stream) {
    if (!seq_lens || !page_table || !shared_len || !page_ok(page_size) || max_seq_len < 0) return TOPK_EINVAL;
    if (num_shared_pages < 0 || (num_shared_pages > 0 && !shared_pages)) return TOPK_EINVAL;
    if (page_table_stride < (static_cast<int64_t>(max_seq_len) + page_size - 1) / page_size || page_table_stride < 1)
        return TOPK_EINVAL;
    if (misaligned(shared_pages, 4) || misaligned(shared_len, 4)) return TOPK_EALIGN;
    const int64_t room = static_cast<int64_t>(num_shared_pages) * page_size;
    LatentParams p = {};
    p.q = q;
    p.q_row_stride = q_row_stride;
    p.q_query_stride = q_query_stride;
    p.q_head_stride = q_head_stride;
    p.cache = cache;
    p.slot_stride = slot_stride;
    p.num_slots = num_slots;
    p.seq_lens = seq_lens;
    p.table = page_table;
    p.table_stride = page_table_stride;
    p.log2_page = log2_of(page_size);
    p.max_len = max_seq_len;
    p.batch = batch;
    p.queries = queries;
    p.heads = heads;
    p.scale = scale;
    p.out = out;
    p.lse = lse_or_null;
    p.workspace = workspace;
    p.shared_pages = shared_pages;
    p.shared_len = shared_len;
    p.max_shared = static_cast<int32_t>(room < max_seq_len ? room : max_seq_len);
    const topk_status_t st = check_latent(p, dtype, topk_attend_shared_workspace_bytes(batch, queries, heads), workspace_bytes);
    return st == TOPK_OK ? run_latent(p, dtype, reinterpret_cast<cudaStream_t>(stream)) : st;
}

topk_status_t topk_attend_prompt(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_nope,
                                 int64_t k_token_stride, int64_t k_head_stride, const void* k_rope,
                                 int64_t k_rope_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                                 const int32_t* cu_q, const int32_t* cu_k, int32_t batch, int32_t total_q,
                                 int32_t total_k, int32_t heads, float scale, int32_t causal, topk_dtype_t dtype,
                                 void* out, float* lse_or_null, topk_stream_t stream) {
    if (batch < 1 || heads < 1 || total_q < 0 || total_k < 0 || !dtype_ok(dtype) || std::isnan(scale) || !cu_q || !cu_k)
        return TOPK_EINVAL;
    if ((total_q > 0 && (!q || !out)) || (total_k > 0 && (!k_nope || !k_rope || !v))) return TOPK_EINVAL;
    if (static_cast<int64_t>(total_q) * heads > kMaxQueryHeads) return TOPK_EINVAL;
    if (!token_stride_ok(q_token_stride, kNope + kRope, total_q) || !token_stride_ok(k_token_stride, kNope, total_k) ||
        !token_stride_ok(k_rope_stride, kRope, total_k) || !token_stride_ok(v_token_stride, kValue, total_k) ||
        !row_stride_ok(q_head_stride, 0) || !row_stride_ok(k_head_stride, 0) || !row_stride_ok(v_head_stride, 0))
        return TOPK_EINVAL;
    if (misaligned(q, 16) || misaligned(k_nope, 16) || misaligned(k_rope, 16) || misaligned(v, 16) ||
        misaligned(out, 32) || misaligned(lse_or_null, 4) || misaligned(cu_q, 4) || misaligned(cu_k, 4) ||
        q_token_stride % 8 || q_head_stride % 8 || k_token_stride % 8 || k_head_stride % 8 || k_rope_stride % 8 ||
        v_token_stride % 8 || v_head_stride % 8)
        return TOPK_EALIGN;
    AttendDevice device;
    const topk_status_t st = attend_device(&device);
    if (st != TOPK_OK) return st;
    if (total_q == 0) return TOPK_OK;
    PromptParams p = {q,      q_token_stride, q_head_stride, k_nope, k_token_stride, k_head_stride, k_rope,
                      k_rope_stride, v,       v_token_stride, v_head_stride, cu_q,   cu_k,          batch,
                      total_q, total_k, heads, scale,        causal, out,            lse_or_null,   wait_limit()};
    return launch_prompt(p, dtype, device, reinterpret_cast<cudaStream_t>(stream));
}

topk_status_t topk_read_attend_flags(uint32_t* flags_host, int32_t clear, topk_stream_t stream) {
    if (!flags_host) return TOPK_EINVAL;
    AttendDevice device;
    const topk_status_t st = attend_device(&device);
    if (st != TOPK_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(flags_host, device.flags, sizeof(uint32_t), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess && clear) e = cudaMemsetAsync(device.flags, 0, sizeof(uint32_t), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return e == cudaSuccess ? TOPK_OK : api_cuda_fail(e, "attention flags");
}

}  // extern "C"
