// attend_prompt.cu -- expanded latent attention for prompts (ragged, causal or
// not) on the tensor cores.
//
// Mathematics: o = sum_j p_j v_j, p = softmax(scale (q_n.k_n + q_r.k_r)), with a
// running reference m and sum l per query: a tile of keys adds
// 2^(x_j - m) v_j, x = scale log2(e) s, and when a tile's maximum has passed m
// by far enough (kHead and kLag of tc.cuh say how far, and what the two-byte
// weights are off by) the sums so far are multiplied by 2^(m - m').  The rotary part is
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
// One block per SM takes pieces of work in turn, so that the next piece's
// queries, keys and first scores are under way while this one's results are
// written (a block a piece: 469 us where this took 455, and 103 where it took 99,
// on the two cases below).
//
// Measured: a prompt of 8192 tokens, 32 heads, causal 459 to 474 us, 1.45 to 1.50
// PFLOP/s (75 to 78 % of the measured burst rate, 84 to 87 % of the sustained
// one, at the power limit); 8 pieces of up to 1024 tokens after up to 4096
// cached ones, 16 heads 95 to 106 us.  A
// step takes 3150 cycles for 2560 of products: the first product reads 128 bytes a
// cycle from shared memory, all there is, beside the copies' writes (92 cycles in
// place of 64).  Pairs of blocks with products of M = 256, which read less, were 3 %
// faster on the one prompt and 14 % slower on the pieces (blocks of 512 queries).
//
// With few pieces of work and long keys the blocks of a cluster share a piece:
// each takes a range of its keys, and the sums are joined through the cluster's
// shared memory, a row's parts in the order of the keys (one query of 16 heads on
// 8192 keys: 115 us by a block a piece, 32 by six).
//
// Warps: 0-3 and 4-7 softmax of tile 0 and 1 (one query a thread), 8 products,
// 9 copies, 10 finds the next piece of work.  The second product starts on the
// first half of a step's weights while the second half is being computed.
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
constexpr int kThreads = 352;
constexpr uint32_t kColumns = 512;
constexpr int kMaxSplit = 8;   // blocks of a cluster
// Up to 4 steps are not shared (8 heads of 512 tokens: 16.4 us alone, 18.4 in two
// parts); longer ones are, in parts of 2 steps or more (4 requests of 64 queries
// on 1024 keys: 22.5 us alone, 18.4 in parts of 4 steps, 16.4 in parts of 2).
constexpr int kAloneSteps = 4, kLeastSteps = 2;

struct PromptMaps {
    CUtensorMap q, k_nope, k_rope, v;
};

// A piece of work: 256 queries of one head and, in a cluster that shares it, a
// range of its keys: those from range.z on, as many steps as `most`.
struct Item {
    int4 range;     // the request's first query, the end of its queries, the same of its keys
    int32_t block;  // of the request's queries, -1: there is no more work
    int32_t head;
    int32_t most, parts;  // blocks that share it

    __device__ __forceinline__ int first(int t) const { return range.x + block * kBlockRows + t * kTile; }  // query of tile t
    __device__ __forceinline__ int keys() const { return range.w - range.z; }
    // Keys seen by query i (of the whole tensor): all, or all but those after it.
    __device__ __forceinline__ int seen(bool causal, int i) const {
        return causal ? max(keys() - (range.y - 1 - i), 0) : keys();
    }
    __device__ __forceinline__ int steps(bool causal, int t) const {
        const int last = min(first(t) + kTile, range.y) - 1;
        return last < first(t) ? 0 : min((seen(causal, last) + kTile - 1) / kTile, most);
    }
};

// By one warp: the block of queries with a number.  Blocks are numbered through
// the requests, ceil(queries / 256) each.  Offsets below an earlier one count
// as that one, so requests never overlap.  Up to 32 requests are taken by
// falling number of keys, so that the last blocks are short ones (8 requests
// of 1 to 5120 keys: 123 -> 107 us when this was added); more as they come.
__device__ __forceinline__ void find(const PromptParams& p, int lane, int index, int4& range, int& block) {
    block = -1;
    range = {};
    bool found = false;
    int before = 0;
    int q_upto = min(max(p.cu_q[0], 0), p.total_q), k_upto = min(max(p.cu_k[0], 0), p.total_k);
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
}

struct Barriers {
    uint64_t key_full[2], key_empty[2], value_full[2], value_empty[2];  // by step mod 2
    uint64_t query_full[2], query_empty[2];
    uint64_t item_full[2], item_empty[2];
    uint64_t score[2], weight[2][2], sum[2];  // weights by tile and half of the step's keys
    uint64_t end;
    uint32_t tmem;
    uint32_t gave_up;
    Item item[2];  // this piece of work and the next
    int3 kept[8];  // by softmax warp: the tile's first query, the end of the queries, the head
};
constexpr int kSmem = 6 * kPiece + kRing * kPiece + static_cast<int>(sizeof(Barriers)) + 1024;

// All threads of a cluster whose blocks have taken a part of the same piece of
// work each.  The parts' sums go to shared memory (queries, keys and values are
// not needed any more) as [128 / 4][256 rows] float4 and (maximum, sum) by row;
// then each thread of the first eight warps joins 16 values of a row at a time,
// taken in turn by the whole cluster.
template <bool kBf16>
__device__ __forceinline__ void join(const PromptParams& p, const Item& w, uint32_t base, uint32_t sums, float m, float l,
                                     int split) {
    const int warp = threadIdx.x >> 5, rows = min(w.range.y - w.first(0), kBlockRows);
    const uint32_t stats = base + kBlockRows * kValue * 4;
    if (warp < 8 && (warp << 5) < rows) {
        const uint32_t from = sums + (static_cast<uint32_t>(warp & 3) << 21) + (warp >> 2) * kValue;
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(stats + 8 * threadIdx.x), "f"(m), "f"(l) : "memory");
        if (w.steps(p.causal, warp >> 2)) {
#pragma unroll 1
            for (int c = 0; c < kValue / 32; ++c) {
                uint32_t o[32];
                tc::load32(from + 32 * c, o);
                tc::wait_load();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    ptx::sts_u4(base + ((8 * c + i) * kBlockRows + threadIdx.x) * 16,
                                make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
            }
        }
    }
    __syncwarp();
    ptx::cluster_sync();
    constexpr int kColumns = kValue / 16;
    const int rank = static_cast<int>(ptx::cluster_ctarank());
    if (warp < 8)
        for (int unit = rank * 256 + static_cast<int>(threadIdx.x); unit < rows * kColumns; unit += split * 256) {
            const int r = unit % rows, c = unit / rows;
            float2 part[kMaxSplit];
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < kMaxSplit; ++i)
                if (i < w.parts) {
                    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                                 : "=f"(part[i].x), "=f"(part[i].y)
                                 : "r"(ptx::map_rank(stats + 8 * r, i)));
                    top = fmaxf(top, part[i].x);
                }
            const float shift = top == -INFINITY ? 0.f : top;
            float sum = 0.f, o[16] = {};
#pragma unroll
            for (int i = 0; i < kMaxSplit; ++i) {
                if (i >= w.parts || part[i].y == 0.f) continue;  // a part that saw nothing
                const uint32_t at = ptx::map_rank(base + (4 * c * kBlockRows + r) * 16, i);
                const float by = exp2f(part[i].x - shift);
                sum += part[i].y * by;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 x = ptx::ld_cluster_v4(at + k * kBlockRows * 16);
                    o[4 * k] += __uint_as_float(x.x) * by;
                    o[4 * k + 1] += __uint_as_float(x.y) * by;
                    o[4 * k + 2] += __uint_as_float(x.z) * by;
                    o[4 * k + 3] += __uint_as_float(x.w) * by;
                }
            }
            const float by = sum == 0.f ? 0.f : 1.f / sum;
            const int64_t at = static_cast<int64_t>(w.first(0) + r) * p.heads + w.head;
            uint32_t pairs[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) pairs[k] = tc::pack<kBf16>(o[2 * k] * by, o[2 * k + 1] * by);
            tc::store_v8(static_cast<uint16_t*>(p.out) + at * kValue + 16 * c, pairs);
            if (p.lse && c == 0) p.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
        }
    __syncwarp();
    ptx::cluster_sync();  // no block ends while others read its parts
}

// kSplit: each cluster of `split` blocks takes one piece of work.
template <bool kBf16, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const PromptParams p, const __grid_constant__ PromptMaps maps, uint32_t* flags, float scale_log2,
                  bool negate, int split) {
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

    if (warp == 0) {
        if (lane == 0) {
            bar.gave_up = p.wait.none;
            for (int t = 0; t < 2; ++t) {
                ptx::mbar_init(&bar.key_full[t], 1);
                ptx::mbar_init(&bar.key_empty[t], 1);
                ptx::mbar_init(&bar.value_full[t], 1);
                ptx::mbar_init(&bar.value_empty[t], 1);
                ptx::mbar_init(&bar.query_full[t], 1);
                ptx::mbar_init(&bar.query_empty[t], 1);
                ptx::mbar_init(&bar.item_full[t], 1);
                ptx::mbar_init(&bar.item_empty[t], 10);
                ptx::mbar_init(&bar.score[t], 1);
                ptx::mbar_init(&bar.weight[t][0], 4);
                ptx::mbar_init(&bar.weight[t][1], 4);
                ptx::mbar_init(&bar.sum[t], 1);
            }
            ptx::mbar_init(&bar.end, 1);
            ptx::fence_mbarrier_init();
        }
    }
    if (warp == 8) tc::alloc<1>(ptx::smem_addr(&bar.tmem), kColumns);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = bar.tmem;
    const tc::Waits wait{&bar.gave_up, p.wait.ns};

    // The warps that copy, multiply and compute take the same pieces of work,
    // each at its own time: copies for the next begin while the last results of
    // this one are being written.
    const auto take = [&](int k, Item& item) {  // by a whole warp; false: there is no more
        if (!wait.all(&bar.item_full[k & 1], (k >> 1) & 1)) return false;
        item = bar.item[k & 1];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bar.item_empty[k & 1]);
        return !wait.over() && item.block >= 0;
    };

    float m_part = -INFINITY, l_part = 0.f;  // what a softmax thread brings to the join
    if (warp == 10) {
        // Pieces are dealt out in turn, every other round backwards, so that
        // no block gets the longest of each.
        for (int k = 0;; ++k) {
            if (k >= 2 && !wait.all(&bar.item_empty[k & 1], ((k >> 1) - 1) & 1)) break;
            const int takers = static_cast<int>(gridDim.x) / split, taker = static_cast<int>(blockIdx.x) / split;
            const int in_round = k & 1 ? takers - 1 - taker : taker;
            const int64_t number = static_cast<int64_t>(k) * takers + in_round, index = number / p.heads;
            int4 range;
            int block = -1;
            if ((!kSplit || k == 0) && index <= p.total_q) find(p, lane, static_cast<int>(index), range, block);
            Item item = {range, block, static_cast<int32_t>(number % p.heads), INT32_MAX, 1};
            if (kSplit && block >= 0) {
                const int rank = static_cast<int>(blockIdx.x) % split;
                const int steps = max(item.steps(p.causal, 0), item.steps(p.causal, 1));
                item.parts = steps > kAloneSteps ? min(split, (steps + kLeastSteps - 1) / kLeastSteps) : 1;
                item.most = (steps + item.parts - 1) / item.parts;
                item.range.z = static_cast<int32_t>(
                    min(static_cast<int64_t>(range.z) + static_cast<int64_t>(rank) * item.most * kTile, static_cast<int64_t>(range.w)));
                if (rank >= item.parts) {
                    item.most = 0;  // joins in the join only
                    if (item.parts == 1) item.block = -1;
                }
            }
            if (lane == 0) {
                bar.item[k & 1] = item;
                ptx::mbar_arrive(&bar.item_full[k & 1]);
            }
            __syncwarp();
            if (item.block < 0 || wait.over()) break;
        }
    } else if (warp == 9) {
        // The ring's pieces i - 8 must have been used before pieces i are
        // filled: whole groups are waited for, the keys or the values of
        // the step in which they were.
        // Once a wait of the block has given up, the products announce what
        // they did not wait for (a condition on them cost 2 % of a long
        // prompt), with the flag set before: nothing is copied after it.
        const auto free_by = [&](uint64_t* empty, uint32_t parity) { return wait(empty, parity) && !*wait.gave_up; };
        const auto room = [&](int last) {
            const int used = last - kRing;
            if (used < 0) return true;
            const int step = used / kStepPieces;
            return free_by(used % kStepPieces < kKeyPieces ? &bar.key_empty[step & 1] : &bar.value_empty[step & 1],
                           (step >> 1) & 1);
        };
        int key_steps = 0, value_steps = 0, loaded[2] = {0, 0};
        Item w;
        for (int k = 0; take(k, w); ++k) {
            if (lane == 0) {
                const int steps[2] = {w.steps(p.causal, 0), w.steps(p.causal, 1)}, n = max(steps[0], steps[1]);
                const int q_head = p.q_head_stride ? w.head : 0, k_head = p.k_head_stride ? w.head : 0,
                          v_head = p.v_head_stride ? w.head : 0;
                const auto load_queries = [&](int t) {
                    if (loaded[t] > 0 && !free_by(&bar.query_empty[t], (loaded[t] - 1) & 1)) return false;
                    ptx::mbar_arrive_expect_tx(&bar.query_full[t], 3 * kPiece);
                    for (int c = 0; c < 3; ++c)
                        tc::load_3d(queries + (3 * t + c) * kPiece, &maps.q, 64 * c, q_head, w.first(t),
                                    &bar.query_full[t]);
                    ++loaded[t];
                    return true;
                };
                const bool on = steps[0] == 0 || load_queries(0);
                for (int j = 0; j < n && on; ++j) {
                    const int row = w.range.z + j * kTile, step = key_steps, piece = step * kStepPieces;
                    const auto at = [&](int i) { return ring + (piece + i) % kRing * kPiece; };
                    if (!room(piece) || !room(piece + 2)) break;
                    uint64_t* full = &bar.key_full[step & 1];
                    ptx::mbar_arrive_expect_tx(full, kKeyPieces * kPiece);
                    for (int c = 0; c < 2; ++c) tc::load_3d(at(c), &maps.k_nope, 64 * c, k_head, row, full);
                    tc::load_2d(at(2), &maps.k_rope, 0, row, full);
                    ++key_steps;
                    if (j == 0 && steps[1] && !load_queries(1)) break;
                    if (!room(piece + 3) || !room(piece + 4)) break;
                    full = &bar.value_full[step & 1];
                    ptx::mbar_arrive_expect_tx(full, 2 * kPiece);
                    for (int c = 0; c < 2; ++c)  // 64 keys by 128 values
                        for (int d = 0; d < 2; ++d)
                            tc::load_3d(at(3 + c) + d * (kPiece / 2), &maps.v, 64 * d, v_head, row + 64 * c, full);
                    ++value_steps;
                }
            }
            __syncwarp();
        }
        if (lane == 0) {  // what is in flight lands before the block ends
            for (int i = max(0, key_steps - 2); i < key_steps; ++i) tc::Waits::drain(&bar.key_full[i & 1], (i >> 1) & 1);
            for (int i = max(0, value_steps - 2); i < value_steps; ++i)
                tc::Waits::drain(&bar.value_full[i & 1], (i >> 1) & 1);
            for (int t = 0; t < 2; ++t)
                if (loaded[t]) tc::Waits::drain(&bar.query_full[t], (loaded[t] - 1) & 1);
        }
    } else if (warp == 8) {
        const uint32_t score_instr = tc::instruction(kBf16, kTile, kTile, negate, false);
        const uint32_t sum_instr = tc::instruction(kBf16, kTile, kValue, false, true);
        const uint64_t query_at = tc::operand(queries), key_at = tc::operand(ring), value_at = tc::operand(ring, kPiece / 2);
        int base = 0, done[2] = {0, 0}, loaded[2] = {0, 0};  // steps of the work before, in all and by tile; queries
        int steps[2] = {0, 0};
        const auto scores = [&](int t, int j) {  // and, after the second tile's, the keys are free
            if (j == 0) wait.warp(&bar.query_full[t], loaded[t]++ & 1);
            const int step = base + j, piece = step * kStepPieces;
            wait.warp(&bar.key_full[step & 1], (step >> 1) & 1);
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
                if (t == 1 || j >= steps[1]) tc::commit<1>(&bar.key_empty[step & 1]);
                if (j == steps[t] - 1) tc::commit<1>(&bar.query_empty[t]);
            }
            __syncwarp();
        };
        const auto sums = [&](int t, int j, int half) {
            wait.warp(&bar.weight[t][half], (done[t] + j) & 1);
            tc::fence_after();
            const int step = base + j;
            const uint64_t b = value_at + (step * kStepPieces + kKeyPieces + half) % kRing * (kPiece >> 4);
            if (tc::elect()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc::mma_tmem(tmem + 256 + t * kValue, tmem + t * kTile + 32 * half + 8 * k, b + 128 * k, sum_instr,
                                 j > 0 || half > 0 || k > 0);
                if (half == 1) {
                    tc::commit<1>(&bar.sum[t]);
                    if (t == 1 || j >= steps[1]) tc::commit<1>(&bar.value_empty[step & 1]);
                }
            }
            __syncwarp();
        };
        Item w;
        for (int k = 0; take(k, w); ++k) {
            steps[0] = w.steps(p.causal, 0);
            steps[1] = w.steps(p.causal, 1);
            const int n = max(steps[0], steps[1]);
            // The first tile may see one step less than the second (causal), or
            // the second have no queries; so the last of the two in a step frees
            // its keys and values.
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (steps[t]) scores(t, 0);
            for (int j = 0; j < n; ++j) {
                const int step = base + j;
                wait.warp(&bar.value_full[step & 1], (step >> 1) & 1);
                const int left = w.keys() - j * kTile;
                if (left < kTile) {
                    // Rows past the request's keys belong to others or to nobody
                    // and may hold anything: a weight of zero would not hide a NaN.
                    for (int i = left * 16 + lane; i < kTile * 16; i += 32) {
                        const int row = i >> 4, piece = (step * kStepPieces + kKeyPieces + (row >> 6)) % kRing;
                        ptx::sts_u4(ring + piece * kPiece + ((i >> 3) & 1) * (kPiece / 2) + (row & 63) * 128 + (i & 7) * 16,
                                    make_uint4(0, 0, 0, 0));
                    }
                    tc::fence_async();
                    __syncwarp();
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (j < steps[t]) {
                        sums(t, j, 0);
                        sums(t, j, 1);
                    }
                    if (j + 1 < steps[t]) scores(t, j + 1);
                }
            }
            base += n;
#pragma unroll
            for (int t = 0; t < 2; ++t) done[t] += steps[t];
        }
        if (tc::elect()) {
            tc::commit<1>(&bar.end);
            tc::Waits::drain(&bar.end, 0);
        }
        __syncwarp();
    } else if (warp < 8) {
        const int t = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        const uint32_t score = lanes + t * kTile, sums = lanes + 256 + t * kValue;
        int done = 0;  // steps of the work before
        for (int k = 0; !kSplit || k < 1; ++k) {
            int steps, limit;
            {
                Item w;
                if (!take(k, w)) break;
                const int query = w.first(t) + row;
                steps = w.steps(p.causal, t);
                limit = query < w.range.y ? w.seen(p.causal, query) : 0;
                // Needed again at the end; the registers are full until then.
                if (lane == 0) bar.kept[warp] = make_int3(w.first(t), w.range.y, w.head);
                __syncwarp();
            }
            float m = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int j = 0; j < steps; ++j) {
                wait.warp(&bar.score[t], (done + j) & 1);
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
                const bool raise = tile_top > m + (tc::kHead<kBf16> + tc::kLag) || (m == -INFINITY && tile_top > m);
                if (__any_sync(~0u, raise)) {
                    const float next = raise ? tile_top - tc::kHead<kBf16> : m;
                    const float by = raise ? tc::exp2_approx(m - next) : 1.f;
                    m = next;
                    l *= by;
                    if (j > 0) {
                        wait.warp(&bar.sum[t], (done + j - 1) & 1);
                        tc::fence_after();
#pragma unroll 1
                        for (int c = 0; c < kValue / 8; ++c) {
                            uint32_t o[8];
                            tc::load8(sums + 8 * c, o);
                            tc::wait_load();
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
                            tc::store8(sums + 8 * c, o);
                        }
                    }
                }
                const float shift = m == -INFINITY ? 0.f : -m;
                const float2 scale2 = make_float2(scale_log2, scale_log2), shift2 = make_float2(shift, shift);
                float2 add[2] = {};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pairs[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float2 x = tc::fma2(make_float2(s[64 * half + 2 * i], s[64 * half + 2 * i + 1]), scale2, shift2);
                        x = make_float2(tc::exp2_approx(x.x), tc::exp2_approx(x.y));
                        add[i & 1] = tc::add2(add[i & 1], x);
                        pairs[i] = tc::pack<kBf16>(x.x, x.y);
                    }
                    tc::store32(score + 32 * half, pairs);
                    tc::wait_store();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&bar.weight[t][half]);
                }
                l += (add[0].x + add[0].y) + (add[1].x + add[1].y);
            }
            if (steps) {
                wait.warp(&bar.sum[t], (done + steps - 1) & 1);
                tc::fence_after();
            }
            if (kSplit && bar.item[0].parts > 1) {
                m_part = m;
                l_part = l;
                break;
            }
            const int3 kept = bar.kept[warp];
            __syncwarp();
            const int query = kept.x + (threadIdx.x & 127);
            const bool real = query < kept.y;
            const float by = l == 0.f ? 0.f : 1.f / l;
            const int64_t at = static_cast<int64_t>(query) * p.heads + kept.z;
            uint16_t* out = static_cast<uint16_t*>(p.out) + at * kValue;
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
                uint32_t o[64];  // (of a tile without steps: not used)
                tc::load32(sums + 64 * c, o);
                tc::load32(sums + 64 * c + 32, o + 32);
                tc::wait_load();
                if (real) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t pairs[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float a = __uint_as_float(o[16 * i + 2 * k]) * by, b = __uint_as_float(o[16 * i + 2 * k + 1]) * by;
                            pairs[k] = l == 0.f ? 0u : tc::pack<kBf16>(a, b);
                        }
                        tc::store_v8(out + 64 * c + 16 * i, pairs);
                    }
                }
                __syncwarp();
            }
            if (p.lse && real) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            tc::fence_before();
            done += steps;
        }
    }
    __syncthreads();
    if (kSplit && bar.item[0].parts > 1) {  // the same for all blocks of a cluster
        tc::fence_after();
        join<kBf16>(p, bar.item[0], base, tmem + 256, m_part, l_part, split);
        tc::fence_before();
        __syncthreads();
    }
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

    // Each request with queries has at most (queries + 255) / 256 blocks.
    const int64_t requests = p.batch < p.total_q ? p.batch : p.total_q;
    const int64_t most = p.heads * ((p.total_q + (kBlockRows - 1) * requests) / kBlockRows);
    const auto kernel = bf16 ? prompt_kernel<true, false> : prompt_kernel<false, false>;
    const auto split_kernel = bf16 ? prompt_kernel<true, true> : prompt_kernel<false, true>;
    static std::atomic<bool> prepared[2][2][AttendDevice::kMax];
    cudaError_t e = cudaSuccess;
    // As many blocks a piece as leave all clusters on the device at once (15 of
    // 8 blocks, 23 of 6, 36 of 4, 76 of 2), if a request can have keys for them.
    int split = 1;
    if (2 * most <= device.sms && p.total_k > kAloneSteps * kTile) {
        static std::atomic<int> fitting[2][kMaxSplit + 1][AttendDevice::kMax];  // clusters, plus 1; 0: not known yet
        e = allow_shared(split_kernel, kSmem, prepared[bf16][1][device.index]);
        for (int n = kMaxSplit; e == cudaSuccess && split == 1 && n > 1; --n) {
            std::atomic<int>& known = fitting[bf16][n][device.index];
            int fit = known.load(std::memory_order_relaxed) - 1;
            if (fit < 0) {
                e = clusters_at_once(&fit, split_kernel, kThreads, kSmem, n);
                if (e == cudaSuccess) known.store(fit + 1, std::memory_order_relaxed);
            }
            if (e == cudaSuccess && most <= fit) split = n;
        }
    }
    if (e == cudaSuccess && split == 1) e = allow_shared(kernel, kSmem, prepared[bf16][0][device.index]);
    if (e != cudaSuccess) return api_cuda_fail(e, "prompt attention shared memory");
    const unsigned grid = static_cast<unsigned>(split > 1 ? most * split : most < device.sms ? most : device.sms);
    // Scores of a negative scale come from negated queries, so that the
    // largest score is always the largest exponent.
    // A scale of zero becomes the least normal number: hidden scores stay -inf.
    const float scale_log2 = std::fmax(std::fabs(p.scale) * 1.4426950408889634f, FLT_MIN);
    if (split > 1)
        e = launch_early_clusters(split_kernel, dim3(grid), split, kThreads, kSmem, stream, p, maps, device.flags, scale_log2,
                                  p.scale < 0.f, split);
    else
        e = launch_early(kernel, dim3(grid), kThreads, kSmem, stream, p, maps, device.flags, scale_log2, p.scale < 0.f, 1);
    return e == cudaSuccess ? TOPK_OK : api_cuda_fail(e, "prompt attention launch");
}

}  // namespace topkidx
