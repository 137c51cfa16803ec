// serve_tables.cu -- topk_block_tables: page-table entries, lengths and slot
// maps of one step from request lengths, in one launch.
//
// Mathematics: two exclusive prefix sums over the requests, of their new
// tokens and of their new pages P(context + new) - P(context), P(n) =
// ceil(n / page_size); output token t then belongs to the last request whose
// sum is <= t, and the i-th new page of request b is entry sum_b + i of the
// free list.
//
// Bound by latency at every size that a step has (8 bytes read per request,
// 12 written per token), so there is one launch and no pass between blocks:
// every block scans all requests itself (4096 at a time, 4 per thread, kept
// as two arrays of sums in shared memory) and writes its own slice of the
// outputs, finding a token's request by bisection in shared memory.
#include <cuda_runtime.h>

#include <cstdint>

#include "attend_internal.h"
#include "ptx.cuh"

namespace topkidx {
namespace {

constexpr int kThreads = 1024;
constexpr int kPer = 4;
constexpr int kChunk = kThreads * kPer;

struct Request {
    int64_t context, total;  // tokens held and tokens after the step, at most what its row holds
    int64_t fresh;           // new tokens
    int32_t have, need;      // pages held, new pages
    uint32_t flags;
};

__device__ __forceinline__ Request load_request(const TablesParams& p, int32_t b) {
    Request r;
    const int32_t c = p.context[b], n = p.fresh[b];
    const int64_t room = static_cast<int64_t>(p.width) << p.log2_page;
    const int64_t page = int64_t{1} << p.log2_page;
    r.flags = (c < 0 || n < 0) ? TOPK_TABLES_NEGATIVE : 0u;
    r.fresh = n > 0 ? n : 0;
    const int64_t ctx = c > 0 ? c : 0;
    if (ctx + r.fresh > room) r.flags |= TOPK_TABLES_ROW_FULL;
    r.context = min(ctx, room);
    r.total = min(ctx + r.fresh, room);
    r.have = static_cast<int32_t>((r.context + page - 1) >> p.log2_page);
    r.need = static_cast<int32_t>((r.total + page - 1) >> p.log2_page) - r.have;
    return r;
}

// The last i in [0, n) with sums[i] <= x (sums does not decrease, sums[0] <= x).
__device__ __forceinline__ int last_not_above(const int32_t* sums, int n, int32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int32_t saturate(int64_t x) {
    return static_cast<int32_t>(min(x, static_cast<int64_t>(INT32_MAX)));
}

__global__ void __launch_bounds__(kThreads, 1) block_tables_kernel(const TablesParams p) {
    extern __shared__ int32_t sums[];
    int32_t* tokens_before = sums;          // [kChunk], from the chunk's start
    int32_t* pages_before = sums + kChunk;  // [kChunk]
    __shared__ int64_t warp_tokens[32], warp_pages[32];
    __shared__ uint32_t all_flags;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t nb = gridDim.x, me = blockIdx.x;
    const int32_t page_mask = static_cast<int32_t>((int64_t{1} << p.log2_page) - 1);
    if (tid == 0) all_flags = 0;
    int64_t token0 = 0, page0 = 0;  // sums before the chunk
    for (int32_t base = 0; base < p.batch; base += kChunk) {
        const int count = min(kChunk, p.batch - base);
        // Sums of this thread's requests, then of the threads before it.
        int64_t t[kPer], g[kPer], ts = 0, gs = 0;
        uint32_t flags = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = tid * kPer + i;
            t[i] = ts;
            g[i] = gs;
            if (at < count) {
                const Request r = load_request(p, base + at);
                ts += r.fresh;
                gs += r.need;
                flags |= r.flags;
            }
        }
        int64_t tx = ts, gx = gs;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t a = __shfl_up_sync(~0u, tx, d), b = __shfl_up_sync(~0u, gx, d);
            if (lane >= d) {
                tx += a;
                gx += b;
            }
        }
        flags = __reduce_or_sync(~0u, flags);
        __syncthreads();  // the chunk before is done with the sums
        if (lane == 31) {
            warp_tokens[warp] = tx;
            warp_pages[warp] = gx;
        }
        if (lane == 0 && flags) atomicOr(&all_flags, flags);
        __syncthreads();
        int64_t tb = 0, gb = 0, tall = 0, gall = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w == warp) {
                tb = tall;
                gb = gall;
            }
            tall += warp_tokens[w];
            gall += warp_pages[w];
        }
        tb += tx - ts;
        gb += gx - gs;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            tokens_before[tid * kPer + i] = saturate(tb + t[i]);
            pages_before[tid * kPer + i] = saturate(gb + g[i]);
        }
        __syncthreads();
        // Lengths and offsets of this block's share of the requests.
        for (int at = static_cast<int>(me) * kThreads + tid; at < count; at += static_cast<int>(nb) * kThreads) {
            p.seq_lens[base + at] = saturate(load_request(p, base + at).total);
            p.cu_new[base + at] = saturate(token0 + tokens_before[at]);
        }
        // New pages.
        for (int64_t i = me * kThreads + tid; i < gall; i += nb * kThreads) {
            const int at = last_not_above(pages_before, count, static_cast<int32_t>(i));
            const Request r = load_request(p, base + at);
            const int64_t from = page0 + i;
            p.table[static_cast<int64_t>(base + at) * p.table_stride + r.have + (i - pages_before[at])] =
                from < p.num_free ? p.free_pages[from] : -1;
        }
        // Slots of the new tokens.
        const int64_t room = min(tall, static_cast<int64_t>(p.max_tokens) - token0);
        for (int64_t i = me * kThreads + tid; i < room; i += nb * kThreads) {
            const int at = last_not_above(tokens_before, count, static_cast<int32_t>(i));
            const Request r = load_request(p, base + at);
            const int64_t pos = max(p.context[base + at], 0) + (i - tokens_before[at]);
            int32_t slot = -1;
            if (pos < r.total) {
                const int32_t col = static_cast<int32_t>(pos >> p.log2_page);
                int32_t page = -1;
                if (col < r.have) {
                    page = p.table[static_cast<int64_t>(base + at) * p.table_stride + col];
                } else {
                    const int64_t from = page0 + pages_before[at] + (col - r.have);
                    if (from < p.num_free) page = p.free_pages[from];
                }
                const int64_t s = (static_cast<int64_t>(page) << p.log2_page) + (pos & page_mask);
                if (page >= 0 && s <= INT32_MAX) slot = static_cast<int32_t>(s);
            }
            const int64_t out = token0 + i;
            p.slots[out] = slot;
            if (p.positions) p.positions[out] = saturate(pos);
            if (p.rows) p.rows[out] = base + at;
        }
        token0 += tall;
        page0 += gall;
    }
    // What is left of the token buffers.
    for (int64_t i = token0 + me * kThreads + tid; i < p.max_tokens; i += nb * kThreads) {
        p.slots[i] = -1;
        if (p.positions) p.positions[i] = -1;
        if (p.rows) p.rows[i] = -1;
    }
    if (me == 0 && tid == 0) {
        p.cu_new[p.batch] = saturate(token0);
        p.status[0] = static_cast<int32_t>(min(page0, static_cast<int64_t>(p.num_free)));
        p.status[1] = static_cast<int32_t>(all_flags | (page0 > p.num_free ? TOPK_TABLES_NO_PAGES : 0u) |
                                           (token0 > p.max_tokens ? TOPK_TABLES_NO_TOKENS : 0u));
    }
}

}  // namespace

cudaError_t launch_block_tables(const TablesParams& p, cudaStream_t stream) {
    const int64_t items = p.max_tokens > p.batch ? p.max_tokens : p.batch;
    int64_t blocks = (items + kChunk - 1) / kChunk;
    if (blocks < 1) blocks = 1;
    if (blocks > 152) blocks = 152;
    return launch_early(block_tables_kernel, dim3(static_cast<unsigned>(blocks)), kThreads, 2 * kChunk * sizeof(int32_t),
                        stream, p);
}

}  // namespace topkidx
