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
// outputs, finding the request of four neighbouring tokens by one bisection in
// shared memory.  32 requests with a token each 8.7 us a call, most of it the
// host's; 4096 requests with 1.05 M tokens in buffers for 1.18 M 11.6 us
// (one token a thread: 15.3 us).
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
    int32_t fresh;           // new tokens
    int32_t have, need;      // pages held, new pages
    uint32_t flags;
};

__device__ __forceinline__ Request make_request(const TablesParams& p, int32_t c, int32_t n) {
    Request r;
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
// Sums of counts that stay at 2^31 - 1 once they reach it: the order of the
// additions does not matter.
__device__ __forceinline__ int32_t add(int32_t a, int32_t b) {
    return static_cast<int32_t>(min(static_cast<uint32_t>(a) + static_cast<uint32_t>(b), static_cast<uint32_t>(INT32_MAX)));
}
__device__ __forceinline__ int32_t scan(int32_t x, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t y = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x = add(x, y);
    }
    return x;
}

// Four values to out[at..at + 4), of which [from, to) exist: at once where
// they all do (at is a multiple of 4) and the array allows it.
__device__ __forceinline__ void put(int32_t* out, bool whole, int64_t at, int64_t from, int64_t to, const int32_t* v) {
    if (!out) return;
    if (whole && at >= from && at + 4 <= to) {
        *reinterpret_cast<int4*>(out + at) = make_int4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at + i >= from && at + i < to) out[at + i] = v[i];
    }
}

__global__ void __launch_bounds__(kThreads, 1) block_tables_kernel(const TablesParams p, bool whole) {
    extern __shared__ int32_t sums[];
    int32_t* tokens_before = sums;          // [kChunk], from the chunk's start
    int32_t* pages_before = sums + kChunk;  // [kChunk]
    __shared__ int32_t warp_tokens[32], warp_pages[32];
    __shared__ uint32_t all_flags;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t nb = gridDim.x, me = blockIdx.x;
    const int32_t page_mask = static_cast<int32_t>((int64_t{1} << p.log2_page) - 1);
    if (tid == 0) all_flags = 0;
    int32_t token0 = 0, page0 = 0;  // sums before the chunk
    for (int32_t base = 0; base < p.batch; base += kChunk) {
        const int count = min(kChunk, p.batch - base);
        // Sums of this thread's requests, then of the threads before it.
        int32_t t[kPer], g[kPer], ts = 0, gs = 0, c[kPer], f[kPer];
        uint32_t flags = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = tid * kPer + i;
            c[i] = at < count ? p.context[base + at] : 0;
            f[i] = at < count ? p.fresh[base + at] : 0;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const Request r = make_request(p, c[i], f[i]);
            t[i] = ts;
            g[i] = gs;
            ts = add(ts, r.fresh);
            gs = add(gs, r.need);
            flags |= r.flags;
        }
        const int32_t tx = scan(ts, lane), gx = scan(gs, lane);
        flags = __reduce_or_sync(~0u, flags);
        __syncthreads();  // the chunk before is done with the sums
        if (lane == 31) {
            warp_tokens[warp] = tx;
            warp_pages[warp] = gx;
        }
        if (lane == 0 && flags) atomicOr(&all_flags, flags);
        __syncthreads();
        const int32_t tw = scan(warp_tokens[lane], lane), gw = scan(warp_pages[lane], lane);
        const int32_t tall = __shfl_sync(~0u, tw, 31), gall = __shfl_sync(~0u, gw, 31);
        int32_t tb = __shfl_sync(~0u, tw, max(warp - 1, 0)), gb = __shfl_sync(~0u, gw, max(warp - 1, 0));
        if (warp == 0) tb = gb = 0;
        const int32_t tp = __shfl_up_sync(~0u, tx, 1), gp = __shfl_up_sync(~0u, gx, 1);
        if (lane > 0) {
            tb = add(tb, tp);
            gb = add(gb, gp);
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            tokens_before[tid * kPer + i] = add(tb, t[i]);
            pages_before[tid * kPer + i] = add(gb, g[i]);
        }
        __syncthreads();
        // Lengths and offsets of this block's share of the requests.
        for (int at = static_cast<int>(me) * kThreads + tid; at < count; at += static_cast<int>(nb) * kThreads) {
            p.seq_lens[base + at] = saturate(make_request(p, p.context[base + at], p.fresh[base + at]).total);
            p.cu_new[base + at] = add(token0, tokens_before[at]);
        }
        // New pages.
        for (int64_t i = me * kThreads + tid; i < gall; i += nb * kThreads) {
            const int at = last_not_above(pages_before, count, static_cast<int32_t>(i));
            const Request r = make_request(p, p.context[base + at], p.fresh[base + at]);
            const int64_t from = page0 + i;
            p.table[static_cast<int64_t>(base + at) * p.table_stride + r.have + (i - pages_before[at])] =
                from < p.num_free ? p.free_pages[from] : -1;
        }
        // Slots of the new tokens, four neighbours a thread: one bisection, and
        // a page looked up once while they stay in it.
        const int64_t end = min(static_cast<int64_t>(token0) + tall, static_cast<int64_t>(p.max_tokens));
        for (int64_t i0 = token0 / 4 + me * kThreads + tid; 4 * i0 < end; i0 += nb * kThreads) {
            const int64_t t0 = 4 * i0;
            int at = last_not_above(tokens_before, count, static_cast<int32_t>(max(t0 - token0, int64_t{0})));
            int32_t ctx = p.context[base + at];
            Request r = make_request(p, ctx, p.fresh[base + at]);
            int32_t page = -1, page_col = -1, slots[4], positions[4], rows[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t i = t0 + k - token0;
                slots[k] = positions[k] = rows[k] = -1;
                if (i < 0 || t0 + k >= end) continue;
                if (i >= tokens_before[at] + static_cast<int64_t>(r.fresh)) {
                    at = last_not_above(tokens_before, count, static_cast<int32_t>(i));
                    ctx = p.context[base + at];
                    r = make_request(p, ctx, p.fresh[base + at]);
                    page_col = -1;
                }
                const int64_t pos = max(ctx, 0) + (i - tokens_before[at]);
                if (pos < r.total) {
                    const int32_t col = static_cast<int32_t>(pos >> p.log2_page);
                    if (col != page_col) {
                        page = -1;
                        page_col = col;
                        if (col < r.have) {
                            page = p.table[static_cast<int64_t>(base + at) * p.table_stride + col];
                        } else {
                            const int64_t from = static_cast<int64_t>(page0) + pages_before[at] + (col - r.have);
                            if (from < p.num_free) page = p.free_pages[from];
                        }
                    }
                    const int64_t s = (static_cast<int64_t>(page) << p.log2_page) + (pos & page_mask);
                    if (page >= 0 && s <= INT32_MAX) slots[k] = static_cast<int32_t>(s);
                }
                positions[k] = saturate(pos);
                rows[k] = base + at;
            }
            put(p.slots, whole, t0, token0, end, slots);
            put(p.positions, whole, t0, token0, end, positions);
            put(p.rows, whole, t0, token0, end, rows);
        }
        token0 = add(token0, tall);
        page0 = add(page0, gall);
    }
    // What is left of the token buffers.
    const int32_t none[4] = {-1, -1, -1, -1};
    for (int64_t i = token0 / 4 + me * kThreads + tid; 4 * i < p.max_tokens; i += nb * kThreads) {
        put(p.slots, whole, 4 * i, token0, p.max_tokens, none);
        put(p.positions, whole, 4 * i, token0, p.max_tokens, none);
        put(p.rows, whole, 4 * i, token0, p.max_tokens, none);
    }
    if (me == 0 && tid == 0) {
        p.cu_new[p.batch] = token0;
        p.status[0] = min(page0, p.num_free);
        p.status[1] = static_cast<int32_t>(all_flags | (page0 > p.num_free ? TOPK_TABLES_NO_PAGES : 0u) |
                                           (token0 > p.max_tokens ? TOPK_TABLES_NO_TOKENS : 0u));
    }
}

}  // namespace

cudaError_t launch_block_tables(const TablesParams& p, cudaStream_t stream) {
    // Room for four tokens a thread, and a request.
    const int64_t items = p.max_tokens / 4 > p.batch ? p.max_tokens / 4 : p.batch;
    int64_t blocks = (items + kThreads - 1) / kThreads;
    const auto wide = [](const int32_t* x) { return reinterpret_cast<uintptr_t>(x) % 16 == 0; };
    if (blocks < 1) blocks = 1;
    if (blocks > 152) blocks = 152;
    return launch_early(block_tables_kernel, dim3(static_cast<unsigned>(blocks)), kThreads, 2 * kChunk * sizeof(int32_t),
                        stream, p, wide(p.slots) && wide(p.positions) && wide(p.rows));
}

}  // namespace topkidx
