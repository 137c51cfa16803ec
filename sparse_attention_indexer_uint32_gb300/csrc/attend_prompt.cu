// attend_prompt.cu -- expanded latent attention for prompts (ragged, causal or
// not) on the tensor cores.
//
// Mathematics: o = sum_j p_j v_j, p = softmax(scale (q_n.k_n + q_r.k_r)), with a
// running maximum m and sum l per query: a tile of keys adds
// 2^(x_j - m) v_j, x = scale log2(e) s, and when a tile's maximum passes m by
// more than 8 (a factor of 256 that fp32 sums and two-byte weights hold with
// room) the sums so far are multiplied by 2^(m - m').  The rotary part is
// one more 64-wide chunk of the first product, read once for all heads'
// blocks, so keys are never put together in memory.
//
// A block has two tiles of 128 queries of one head and walks the keys 128 at a
// time; the tiles share each load of keys and values.  Its tensor memory is
// full: two score tiles (128 columns each, the weights go back into their
// first 64 as two-byte pairs and are the second product's A operand from
// there) and two sums (128 each).  While one tile's softmax runs, the tensor
// cores work on the other tile.  Shared memory: 96 KB of queries, and a ring of
// eight 16 KB pieces (three of keys and two of values per step).
//
// Measured: a prompt of 8192 tokens, 32 heads, causal 478 us, 1.44 PFLOP/s (75 %
// of the measured burst rate, 84 % of the sustained one, at the power limit); 8
// pieces of up to 1024 tokens after up to 4096 cached ones, 16 heads 104 us.  A
// step takes 3150 cycles for 2560 of products: the first product reads 128 bytes a
// cycle from shared memory, all there is, beside the copies' writes (92 cycles in
// place of 64).  Pairs of blocks with products of M = 256, which read less, were 3 %
// faster on the one prompt and 14 % slower on the pieces (blocks of 512 queries).
//
// Warps: 0-3 and 4-7 softmax of tile 0 and 1 (one query a thread), 8 products,
// 9 copies.  The second product starts on the first half of a step's weights
// while the second half is being computed.
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "attend_internal.h"
#include "tc.cuh"
#include "tensor_map.h"

namespace topkidx {
namespace {

constexpr int kTile = 128;                   // queries a tile, keys a step
constexpr int kBlockRows = 2 * kTile;
constexpr int kPiece = 16384;                // 128 rows of 128 bytes
constexpr int kRing = 8;
constexpr int kKeyPieces = 3, kStepPieces = 5;
constexpr int kThreads = 320;
constexpr uint32_t kColumns = 512;
constexpr float kLag = 8.f;

struct PromptMaps {
    CUtensorMap q, k_nope, k_rope, v;
};

struct Barriers {
    uint64_t key_full[2], key_empty[2], value_full[2], value_empty[2];  // by step mod 2
    uint64_t query[2];
    uint64_t score[2], weight[2][2], sum[2];  // weights by tile and half of the step's keys
    uint64_t end;
    uint32_t tmem;
    uint32_t gave_up;
    int32_t block;  // of the request's
    int4 range;     // its first query, the end of its queries, the same of its keys
};
constexpr int kSmem = 6 * kPiece + kRing * kPiece + static_cast<int>(sizeof(Barriers)) + 1024;

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const PromptParams p, const __grid_constant__ PromptMaps maps, uint32_t* flags, float scale_log2,
                  bool negate) {
    extern __shared__ uint8_t raw[];
    const uint32_t base = (ptx::smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t queries = base, ring = base + 6 * kPiece;
    Barriers& bar = *reinterpret_cast<Barriers*>(raw + (base - ptx::smem_addr(raw)) + (6 + kRing) * kPiece);
    if (threadIdx.x == 0) {
        tc::prefetch_map(&maps.q);
        tc::prefetch_map(&maps.k_nope);
        tc::prefetch_map(&maps.k_rope);
        tc::prefetch_map(&maps.v);
    }
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.heads));
    const int index = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.heads));

    // The request that this block's queries are in: blocks are numbered
    // through the requests, ceil(queries / 256) each.  Offsets below an
    // earlier one count as that one, so requests never overlap.  Up to 32
    // requests are taken by falling number of keys, so that the last blocks
    // are short ones (8 requests of 1 to 5120 keys: 123 -> 107 us); more are
    // taken as they come.
    if (warp == 0) {
        int before = 0;
        bool found = false;
        int block = -1;
        int q_upto = min(max(p.cu_q[0], 0), p.total_q), k_upto = min(max(p.cu_k[0], 0), p.total_k);
        int4 range = {};
        for (int r0 = 0; r0 < p.batch && !found; r0 += 32) {
            const int r = min(r0 + lane, p.batch - 1);
            int q_end = max(min(p.cu_q[r + 1], p.total_q), q_upto), k_end = max(min(p.cu_k[r + 1], p.total_k), k_upto);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int x = __shfl_up_sync(~0u, q_end, d), y = __shfl_up_sync(~0u, k_end, d);
                if (lane >= d) {
                    q_end = max(q_end, x);
                    k_end = max(k_end, y);
                }
            }
            int q_start = __shfl_up_sync(~0u, q_end, 1), k_start = __shfl_up_sync(~0u, k_end, 1);
            if (lane == 0) {
                q_start = q_upto;
                k_start = k_upto;
            }
            // Blocks before this request's: of the requests that come first.
            const int mine = (q_end - q_start + kBlockRows - 1) / kBlockRows, length = k_end - k_start;
            int ahead = 0;
            if (p.batch <= 32) {
#pragma unroll 8
                for (int i = 0; i < 32; ++i) {
                    const int blocks = __shfl_sync(~0u, mine, i), other = __shfl_sync(~0u, length, i);
                    if (other > length || (other == length && i < lane)) ahead += blocks;
                }
            } else {
                int upto = mine;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int x = __shfl_up_sync(~0u, upto, d);
                    if (lane >= d) upto += x;
                }
                ahead = before + upto - mine;
            }
            const unsigned here = __ballot_sync(~0u, index >= ahead && index < ahead + mine);
            if (here) {
                const int at = __ffs(here) - 1;
                found = true;
                // Blocks of a request in falling order: with causal masks the longest first.
                block = __shfl_sync(~0u, mine - 1 - (index - ahead), at);
                range.x = __shfl_sync(~0u, q_start, at);
                range.y = __shfl_sync(~0u, q_end, at);
                range.z = __shfl_sync(~0u, k_start, at);
                range.w = __shfl_sync(~0u, k_end, at);
            }
            before += __reduce_add_sync(~0u, mine);
            q_upto = __shfl_sync(~0u, q_end, 31);
            k_upto = __shfl_sync(~0u, k_end, 31);
        }
        if (lane == 0) {
            bar.range = range;
            bar.block = block;
            bar.gave_up = 0;
            for (int t = 0; t < 2; ++t) {
                ptx::mbar_init(&bar.key_full[t], 1);
                ptx::mbar_init(&bar.key_empty[t], 1);
                ptx::mbar_init(&bar.value_full[t], 1);
                ptx::mbar_init(&bar.value_empty[t], 1);
                ptx::mbar_init(&bar.query[t], 1);
                ptx::mbar_init(&bar.score[t], 1);
                ptx::mbar_init(&bar.weight[t][0], 4);
                ptx::mbar_init(&bar.weight[t][1], 4);
                ptx::mbar_init(&bar.sum[t], 1);
            }
            ptx::mbar_init(&bar.end, 1);
            ptx::fence_mbarrier_init();
        }
    }
    __syncthreads();
    if (bar.block < 0) return;  // more blocks than the requests have

    if (warp == 8) tc::alloc<1>(ptx::smem_addr(&bar.tmem), kColumns);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = bar.tmem;
    const tc::Waits wait{&bar.gave_up};

    const int q0 = bar.range.x, q1 = bar.range.y, k0 = bar.range.z, k1 = bar.range.w;
    const int keys = k1 - k0;
    const int first = q0 + bar.block * kBlockRows;  // first query of tile 0
    // Keys seen by query i (of the whole tensor): all, or all but those after it.
    const auto seen = [&](int i) { return p.causal ? max(keys - (q1 - 1 - i), 0) : keys; };
    int steps[2];
    for (int t = 0; t < 2; ++t) {
        const int last = min(first + (t + 1) * kTile, q1) - 1;
        steps[t] = last < first + t * kTile ? 0 : (seen(last) + kTile - 1) / kTile;
    }
    const int n = max(steps[0], steps[1]);

    if (warp == 9) {
        if (lane == 0) {
            // The ring's pieces i - 8 must have been used before pieces i are
            // filled: whole groups are waited for, the keys or the values of
            // the step in which they were.
            const auto room = [&](int last) {
                const int used = last - kRing;
                if (used < 0) return;
                const int step = used / kStepPieces;
                wait(used % kStepPieces < kKeyPieces ? &bar.key_empty[step & 1] : &bar.value_empty[step & 1], (step >> 1) & 1);
            };
            int key_steps = 0, value_steps = 0;
            const int q_head = p.q_head_stride ? head : 0, k_head = p.k_head_stride ? head : 0,
                      v_head = p.v_head_stride ? head : 0;
            const auto load_queries = [&](int t) {
                ptx::mbar_arrive_expect_tx(&bar.query[t], 3 * kPiece);
                for (int c = 0; c < 3; ++c)
                    tc::load_3d(queries + (3 * t + c) * kPiece, &maps.q, 64 * c, q_head, first + t * kTile, &bar.query[t]);
            };
            if (steps[0]) load_queries(0);
            for (int j = 0; j < n && !bar.gave_up; ++j) {
                const int row = k0 + j * kTile, piece = j * kStepPieces;
                const auto at = [&](int i) { return ring + (piece + i) % kRing * kPiece; };
                room(piece);
                room(piece + 2);
                uint64_t* full = &bar.key_full[j & 1];
                ptx::mbar_arrive_expect_tx(full, kKeyPieces * kPiece);
                for (int c = 0; c < 2; ++c) tc::load_3d(at(c), &maps.k_nope, 64 * c, k_head, row, full);
                tc::load_2d(at(2), &maps.k_rope, 0, row, full);
                ++key_steps;
                if (j == 0 && steps[1]) load_queries(1);
                room(piece + 3);
                room(piece + 4);
                full = &bar.value_full[j & 1];
                ptx::mbar_arrive_expect_tx(full, 2 * kPiece);
                for (int c = 0; c < 2; ++c)  // 64 keys by 128 values
                    for (int d = 0; d < 2; ++d)
                        tc::load_3d(at(3 + c) + d * (kPiece / 2), &maps.v, 64 * d, v_head, row + 64 * c, full);
                ++value_steps;
            }
            if (bar.gave_up) {  // what is in flight lands before the block ends
                for (int i = max(0, key_steps - 2); i < key_steps; ++i) tc::Waits::drain(&bar.key_full[i & 1], (i >> 1) & 1);
                for (int i = max(0, value_steps - 2); i < value_steps; ++i)
                    tc::Waits::drain(&bar.value_full[i & 1], (i >> 1) & 1);
                for (int t = 0; t < 2; ++t)
                    if (steps[t]) tc::Waits::drain(&bar.query[t], 0);
            }
        }
    } else if (warp == 8) {
        const uint32_t score_instr = tc::instruction(kBf16, kTile, kTile, negate, false);
        const uint32_t sum_instr = tc::instruction(kBf16, kTile, kValue, false, true);
        const uint64_t query_at = tc::operand(queries), key_at = tc::operand(ring), value_at = tc::operand(ring, kPiece / 2);
        const auto scores = [&](int t, int j) {  // and, after the second tile's, the keys are free
            if (j == 0) wait.warp(&bar.query[t], 0);
            wait.warp(&bar.key_full[j & 1], (j >> 1) & 1);
            const int piece = j * kStepPieces;
            const uint64_t a = query_at + 3 * t * (kPiece >> 4);
            const uint64_t b[3] = {key_at + piece % kRing * (kPiece >> 4), key_at + (piece + 1) % kRing * (kPiece >> 4),
                                   key_at + (piece + 2) % kRing * (kPiece >> 4)};
            if (tc::elect()) {
#pragma unroll
                for (int c = 0; c < kKeyPieces; ++c)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc::mma<1>(tmem + t * kTile, a + c * (kPiece >> 4) + 2 * k, b[c] + 2 * k, score_instr, (c | k) != 0);
                tc::commit<1>(&bar.score[t]);
                if (t == 1 || j >= steps[1]) tc::commit<1>(&bar.key_empty[j & 1]);
            }
            __syncwarp();
        };
        const auto sums = [&](int t, int j, int half) {
            wait.warp(&bar.weight[t][half], j & 1);
            tc::fence_after();
            const uint64_t b = value_at + (j * kStepPieces + kKeyPieces + half) % kRing * (kPiece >> 4);
            if (tc::elect()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc::mma_tmem(tmem + 256 + t * kValue, tmem + t * kTile + 32 * half + 8 * k, b + 128 * k, sum_instr,
                                 j > 0 || half > 0 || k > 0);
                if (half == 1) {
                    tc::commit<1>(&bar.sum[t]);
                    if (t == 1 || j >= steps[1]) tc::commit<1>(&bar.value_empty[j & 1]);
                }
            }
            __syncwarp();
        };
        // The first tile may see one step less than the second (causal), or
        // the second have no queries; so the last of the two in a step frees
        // its keys and values.
        for (int t = 0; t < 2; ++t)
            if (steps[t]) scores(t, 0);
        for (int j = 0; j < n; ++j) {
            wait.warp(&bar.value_full[j & 1], (j >> 1) & 1);
            const int left = keys - j * kTile;
            if (left < kTile) {
                // Rows past the request's keys belong to others or to nobody
                // and may hold anything: a weight of zero would not hide a NaN.
                for (int i = left * 16 + lane; i < kTile * 16; i += 32) {
                    const int row = i >> 4, piece = (j * kStepPieces + kKeyPieces + (row >> 6)) % kRing;
                    ptx::sts_u4(ring + piece * kPiece + ((i >> 3) & 1) * (kPiece / 2) + (row & 63) * 128 + (i & 7) * 16,
                                make_uint4(0, 0, 0, 0));
                }
                tc::fence_async();
                __syncwarp();
            }
            for (int t = 0; t < 2; ++t) {
                if (j < steps[t]) {
                    sums(t, j, 0);
                    sums(t, j, 1);
                }
                if (j + 1 < steps[t]) scores(t, j + 1);
            }
        }
        if (tc::elect()) {
            tc::commit<1>(&bar.end);
            tc::Waits::drain(&bar.end, 0);
        }
        __syncwarp();
    } else if (warp < 8) {
        const int t = warp >> 2, row = threadIdx.x & 127;
        const int query = first + t * kTile + row;
        const int limit = query < q1 ? seen(query) : 0;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        const uint32_t score = lanes + t * kTile, sums = lanes + 256 + t * kValue;
        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < steps[t]; ++j) {
            wait.warp(&bar.score[t], j & 1);
            tc::fence_after();
            uint32_t raw_s[kTile];
#pragma unroll
            for (int c = 0; c < 4; ++c) tc::load32(score + 32 * c, raw_s + 32 * c);
            tc::wait_load();
            float* s = reinterpret_cast<float*>(raw_s);
            const int left = limit - j * kTile;
            if (__any_sync(~0u, left < kTile)) {
#pragma unroll
                for (int i = 0; i < kTile; ++i)
                    if (i >= left) s[i] = -INFINITY;
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < kTile; i += 2) top[(i >> 1) & 3] = tc::max3(top[(i >> 1) & 3], s[i], s[i + 1]);
            const float tile_top = tc::max3(fmaxf(top[0], top[1]), top[2], top[3]) * scale_log2;
            const bool raise = tile_top > m + kLag || (m == -INFINITY && tile_top > m);
            if (__any_sync(~0u, raise)) {
                const float next = raise ? tile_top : m;
                const float by = raise ? tc::exp2_approx(m - next) : 1.f;
                m = next;
                l *= by;
                if (j > 0) {
                    wait.warp(&bar.sum[t], (j - 1) & 1);
                    tc::fence_after();
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[32];
                        tc::load32(sums + 32 * c, o);
                        tc::wait_load();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
                        tc::store32(sums + 32 * c, o);
                    }
                }
            }
            const float shift = m == -INFINITY ? 0.f : -m;
            const float2 scale2 = make_float2(scale_log2, scale_log2), shift2 = make_float2(shift, shift);
            float2 add[2] = {};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float2 x = tc::fma2(make_float2(s[64 * half + 2 * i], s[64 * half + 2 * i + 1]), scale2, shift2);
                    x = make_float2(tc::exp2_approx(x.x), tc::exp2_approx(x.y));
                    add[i & 1] = tc::add2(add[i & 1], x);
                    w[i] = tc::pack<kBf16>(x.x, x.y);
                }
                tc::store32(score + 32 * half, w);
                tc::wait_store();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bar.weight[t][half]);
            }
            l += (add[0].x + add[0].y) + (add[1].x + add[1].y);
        }
        if (steps[t]) {
            wait.warp(&bar.sum[t], (steps[t] - 1) & 1);
            tc::fence_after();
        }
        const float by = l == 0.f ? 0.f : 1.f / l;
        const int64_t at = static_cast<int64_t>(query) * p.heads + head;
        uint16_t* out = static_cast<uint16_t*>(p.out) + at * kValue;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
            uint32_t o[64];
            if (steps[t]) {
                tc::load32(sums + 64 * c, o);
                tc::load32(sums + 64 * c + 32, o + 32);
                tc::wait_load();
            }
            if (query < q1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float a = __uint_as_float(o[16 * i + 2 * k]) * by, b = __uint_as_float(o[16 * i + 2 * k + 1]) * by;
                        w[k] = l == 0.f ? 0u : tc::pack<kBf16>(a, b);
                    }
                    tc::store_v8(out + 64 * c + 16 * i, w);
                }
            }
            __syncwarp();
        }
        if (p.lse && query < q1) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        tc::fence_before();
    }
    __syncthreads();
    if (warp == 8) {
        tc::fence_after();
        tc::dealloc<1>(tmem, kColumns);
    }
    if (threadIdx.x == 0 && bar.gave_up) atomicOr(flags, TOPK_FLAG_TIMEOUT);
}

}  // namespace

topk_status_t launch_prompt(const PromptParams& p, topk_dtype_t dtype, const AttendDevice& device, cudaStream_t stream) {
    const bool bf16 = dtype == TOPK_BF16;
    PromptMaps maps;
    const auto map3 = [&](CUtensorMap* m, const void* base, int64_t width, int64_t head_stride, int64_t tokens,
                          int64_t token_stride, int rows) {
        // A stride of 0 (all heads alike) is one head for the map; the stride
        // of an extent of one is not used and need not be a legal one.
        const int64_t heads = head_stride ? p.heads : 1;
        const int64_t dims[3] = {width, heads, tokens};
        const int64_t steps[2] = {2 * (heads > 1 ? head_stride : width), 2 * (tokens > 1 ? token_stride : width)};
        return encode_map(m, bf16, base, 3, dims, steps, 2, rows);
    };
    const int64_t rope_dims[2] = {kRope, p.total_k}, rope_step[1] = {2 * (p.total_k > 1 ? p.k_rope_stride : kRope)};
    // Without keys nothing is copied through their maps: any address will do.
    const void* any = p.q;
    CUresult r = map3(&maps.q, p.q, kNope + kRope, p.q_head_stride, p.total_q, p.q_token_stride, kTile);
    if (r == CUDA_SUCCESS)
        r = map3(&maps.k_nope, p.total_k ? p.k_nope : any, kNope, p.k_head_stride, p.total_k, p.k_token_stride, kTile);
    if (r == CUDA_SUCCESS) r = encode_map(&maps.k_rope, bf16, p.total_k ? p.k_rope : any, 2, rope_dims, rope_step, 1, kTile);
    if (r == CUDA_SUCCESS)
        r = map3(&maps.v, p.total_k ? p.v : any, kValue, p.v_head_stride, p.total_k, p.v_token_stride, kTile / 2);
    if (r != CUDA_SUCCESS) return api_cuda_fail(cudaErrorInvalidValue, "prompt attention tensor map");

    const auto kernel = bf16 ? prompt_kernel<true> : prompt_kernel<false>;
    static std::atomic<bool> prepared[2][AttendDevice::kMax];
    cudaError_t e = allow_shared(kernel, kSmem, prepared[bf16][device.index]);
    if (e != cudaSuccess) return api_cuda_fail(e, "prompt attention shared memory");
    // Every request adds at most one block to total / 256.
    const unsigned grid = static_cast<unsigned>(p.heads) *
                          static_cast<unsigned>(p.total_q / kBlockRows + (p.batch < p.total_q ? p.batch : p.total_q));
    // Scores of a negative scale come from negated queries, so that the
    // largest score is always the largest exponent.
    // A scale of zero becomes the least normal number: hidden scores stay -inf.
    const float scale_log2 = std::fmax(std::fabs(p.scale) * 1.4426950408889634f, FLT_MIN);
    e = launch_early(kernel, dim3(grid), kThreads, kSmem, stream, p, maps, device.flags, scale_log2, p.scale < 0.f);
    return e == cudaSuccess ? TOPK_OK : api_cuda_fail(e, "prompt attention launch");
}

}  // namespace topkidx
