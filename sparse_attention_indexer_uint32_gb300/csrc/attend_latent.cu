// attend_latent.cu -- absorbed latent attention over the paged cache, over
// selected slots or whole rows, on the tensor cores.
//
// Mathematics: as in attend_prompt.cu, with one latent row c_j for every head:
// s_hj = q_h.c_j over 576 values, o_h = sum_j p_hj c_j over the first 512.  So a
// row of the cache is read once for up to 128 (query, head) rows of the
// products, 2 * 128 * 1088 operations on 1152 bytes: near the balance of the
// tensor cores and the memory for 128 heads, bound by memory for fewer.
//
// A pair of blocks (a cluster, one per two SMs) takes 128 (query, head) rows
// and walks the slots 128 at a time.  One sum of 128 x 512 in fp32 alone would
// fill an SM's tensor memory, and 128 queries with 128 latent rows its shared
// memory; the pair splits both: products are issued for two SMs at once
// (cta_group::2, M = 128), block r holding the rows 64 r.. of A, half of B and
// the sums of its own rows.  For the first product B is the tile's slots 64 r..
// (all 576 values, K contiguous), for the second the values 256 r.. of all 128
// slots (N contiguous).  The two views overlap in one quarter that cannot be
// shared, because one descriptor serves both blocks: 17/18 of the tile is
// copied to each block (the second time from L2).
//
// Selected slots are copied 16 bytes a thread, four warps per block; a slot that
// is not seen is filled with zeros, so what it holds never meets the sums.
// (Gathers of four rows by the copy engine took 38-57 cycles for 512 bytes and
// bound the kernel at 10400 cycles a tile.)  Pages of 16 slots or more are
// copied by the engine, up to 64 rows of 64 values at a time; the rows past a
// sequence's end are set to zero after they land.  In both cases a warp waits
// for what landed, orders it before the products' reads, and tells the first
// block.
//
// Work is cut in equal runs of tiles, through the rows' ends: the host does not
// know the lengths.  A run's first and last row may be shared with the pairs
// before and after; those write fp32 sums to the workspace and a second kernel
// joins them, in the order of the slots (no atomics: equal calls give equal
// bits).
//
// Warps of each block: 0-3 softmax and results (thread t: row t & 63, slots 64
// (t >> 6).. of the tile, values 256 (t >> 6).. of the sums), 4 products (first
// block only), 5 and 8 copies for the first product, 6 and 9 for the second, 7
// tells of what landed, 10 queries, 11 rows to L2 ahead of their copies.
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

constexpr int kRows = 128;                  // (query, head) rows of a pair
constexpr int kTile = 128;                  // slots a step
constexpr int kHalf = 64;
constexpr int kThreads = 384;
constexpr int kQueryWarp = 10, kPrefetchWarp = 11;
constexpr int kMaxPairs = 80;
constexpr int kKeyPiece = kHalf * 128;      // 64 slots of 64 values
constexpr int kValuePiece = kTile * 128;    // 128 slots of 64 values
constexpr int kPieces = kWidth / 64;        // 9
constexpr int kKeyGroups = 3;               // pieces of keys wait and are freed three at a time
constexpr int kQueryBytes = kPieces * kKeyPiece;
constexpr int kKeyBytes = kPieces * kKeyPiece;
constexpr int kValueBytes = 4 * kValuePiece;
constexpr int kWeightBytes = 2 * kKeyPiece;
constexpr uint32_t kColumns = 512;
constexpr uint32_t kScore = 256;            // column of the two score tiles; the sums have 0..255
constexpr float kLag = 8.f;

struct Shared {
    uint64_t query_full, query_empty;
    // landed: in this block; full: in both (used in the first block).
    uint64_t key_landed[kKeyGroups], key_full[kKeyGroups], key_empty[kKeyGroups];
    uint64_t value_landed[2], value_full[2], value_empty[2];
    uint64_t score[2], weight, sum, end;
    uint64_t mask_full[4];
    uint32_t mask[4][4];
    float exchange[2][kRows];
    uint32_t tmem, gave_up;
    volatile int32_t copied;  // tiles whose first copies are all under way
    int64_t begin, total;  // first tile of this pair's run, tiles of all runs
    int32_t row, tile;     // where the run begins: row of the batch, tile in its group rows
    int64_t scan[kThreads / 32];
};
constexpr int kSmem = kQueryBytes + kKeyBytes + kValueBytes + kWeightBytes + 1024 + 2048;
static_assert(sizeof(Shared) <= 2048, "barriers fit");
static_assert(kSmem <= 232448, "shared memory of a block");

struct LatentMaps {
    CUtensorMap q, cache;
};

__device__ __forceinline__ int length_of(const LatentParams& p, int b) {
    return p.seq_lens ? min(max(p.seq_lens[b], 0), p.max_len) : p.max_len;
}
// Tiles of one group of 128 rows; an empty row has one, all of it hidden.
__device__ __forceinline__ int tiles_of(int length) { return max((length + kTile - 1) / kTile, 1); }
__device__ __forceinline__ int groups_of(const LatentParams& p) { return (p.queries * p.heads + kRows - 1) / kRows; }

// Run of pair i of n: [total i / n, total (i + 1) / n); with fewer tiles than
// pairs the first `total` pairs have one each.
__device__ __forceinline__ int64_t run_start(int64_t total, int i, int n) {
    return total < n ? min(static_cast<int64_t>(i), total) : total * i / n;
}

// All threads of a block: the tiles of the whole batch, and the row of the
// batch in which tile `run_start(total, pair, pairs)` lies, with the tile's
// number from that row's first (the last tile for a pair without a run).
__device__ void locate(const LatentParams& p, int pair, int pairs, int64_t* scan, int64_t* total_out, int64_t* begin_out,
                       int32_t* row_out, int32_t* tile_out) {
    const int threads = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int groups = groups_of(p);
    if (!p.seq_lens) {
        const int64_t each = static_cast<int64_t>(tiles_of(p.max_len)) * groups;
        if (tid == 0) {
            const int64_t total = each * p.batch, begin = run_start(total, pair, pairs);
            const int64_t at = min(begin, total - 1);
            *total_out = total;
            *begin_out = begin;
            *row_out = static_cast<int32_t>(at / each);
            *tile_out = static_cast<int32_t>(at % each);
        }
        __syncthreads();
        return;
    }
    const int per = (p.batch + threads - 1) / threads;
    const int from = min(tid * per, p.batch), to = min(from + per, p.batch);
    int64_t mine = 0;
    for (int b = from; b < to; ++b) mine += static_cast<int64_t>(tiles_of(length_of(p, b))) * groups;
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(~0u, upto, d);
        if (lane >= d) upto += x;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int w = 0; w < threads / 32; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    before += upto - mine;
    const int64_t begin = run_start(total, pair, pairs);
    const int64_t tile = min(begin, total - 1);
    if (tile >= before && tile < before + mine) {
        int64_t at = before;
        int b = from;
        while (true) {
            const int64_t n = static_cast<int64_t>(tiles_of(length_of(p, b))) * groups;
            if (tile < at + n) break;
            at += n;
            ++b;
        }
        *total_out = total;
        *begin_out = begin;
        *row_out = b;
        *tile_out = static_cast<int32_t>(tile - at);
    }
    __syncthreads();
}

// A run's pieces: tiles [first, last) of one group of 128 rows.
struct Segment {
    int row, group, first, last, tiles, length;
};
struct Walk {
    const LatentParams& p;
    int64_t left;
    int row, group, first, groups;

    __device__ Walk(const LatentParams& p, const Shared& sh, int pair, int pairs)
        : p(p), left(run_start(sh.total, pair + 1, pairs) - sh.begin), row(sh.row), groups(groups_of(p)) {
        const int tiles = tiles_of(length_of(p, min(row, p.batch - 1)));
        group = sh.tile / tiles;
        first = sh.tile % tiles;
    }
    __device__ bool next(Segment& s) {
        if (left <= 0) return false;
        s.row = row;
        s.group = group;
        s.length = length_of(p, row);
        s.tiles = tiles_of(s.length);
        s.first = first;
        s.last = static_cast<int>(min(static_cast<int64_t>(s.tiles), first + left));
        left -= s.last - s.first;
        first = 0;
        if (++group == groups) {
            group = 0;
            ++row;
        }
        return true;
    }
};

// Slot of a position, -1 where it is not seen.
template <bool kPaged>
__device__ __forceinline__ int slot_of(const LatentParams& p, int row, int length, int64_t at) {
    if (at >= length) return -1;
    if (!kPaged && p.indices) {
        const int32_t s = p.indices[static_cast<int64_t>(row) * p.indices_stride + at];
        return s < p.num_slots ? s : -1;
    }
    const int pos = static_cast<int>(at);
    const int64_t s = (static_cast<int64_t>(p.table[static_cast<int64_t>(row) * p.table_stride + (pos >> p.log2_page)])
                       << p.log2_page) +
                      (pos & ((1 << p.log2_page) - 1));
    return s >= 0 && s < p.num_slots ? static_cast<int>(s) : -1;
}

// Workspace: what each pair but the first has to join (see Join), then partial
// sums, two places a pair: 0 for a row begun by an earlier pair, 1 for a row
// begun by this pair and finished by a later one.  A place holds the sums as
// [512 / 4][rows] float4, then (maximum, sum) by row: threads hold a row each,
// so neighbouring threads write and read neighbouring addresses.
struct alignas(16) Join {
    int32_t parts;  // parts of the group of rows in which this pair's run is the first to begin, 0: none
    int32_t rows;   // rows of the group
    int64_t at;     // first (query, head) row of the group
};
constexpr size_t kJoinBytes = kMaxPairs * sizeof(Join);
static_assert(kJoinBytes % 16 == 0, "partial sums are aligned");

__device__ __forceinline__ float* part_of(const LatentParams& p, int rows, int place) {
    return reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) + kJoinBytes) +
           static_cast<int64_t>(place) * rows * (kLatent + 2);
}

template <bool kBf16, bool kPaged>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    latent_kernel(const LatentParams p, const __grid_constant__ LatentMaps maps, uint32_t* flags, float scale_log2,
                  bool negate, bool whole_rows, int box_rows) {
    extern __shared__ uint8_t raw[];
    const uint32_t base = (ptx::smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t queries = base, keys = queries + kQueryBytes, values = keys + kKeyBytes,
                   weights = values + kValueBytes;
    Shared& sh = *reinterpret_cast<Shared*>(raw + (weights + kWeightBytes - ptx::smem_addr(raw)));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(ptx::cluster_ctarank());
    const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        sh.gave_up = 0;
        sh.copied = 0;
        ptx::mbar_init(&sh.query_full, 1);
        ptx::mbar_init(&sh.query_empty, 1);
        const uint32_t landings = kPaged ? 1 : 64;
        for (int i = 0; i < kKeyGroups; ++i) {
            ptx::mbar_init(&sh.key_landed[i], landings);
            ptx::mbar_init(&sh.key_full[i], 2);
            ptx::mbar_init(&sh.key_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sh.value_landed[i], landings);
            ptx::mbar_init(&sh.value_full[i], 2);
            ptx::mbar_init(&sh.value_empty[i], 1);
            ptx::mbar_init(&sh.score[i], 1);
        }
        ptx::mbar_init(&sh.weight, 8);
        ptx::mbar_init(&sh.sum, 1);
        ptx::mbar_init(&sh.end, 1);
        for (int i = 0; i < 4; ++i) ptx::mbar_init(&sh.mask_full[i], kPaged ? 1 : 2);
        ptx::fence_mbarrier_init();
    }
    if (warp == 4) tc::alloc<2>(ptx::smem_addr(&sh.tmem), kColumns);
    locate(p, pair, pairs, sh.scan, &sh.total, &sh.begin, &sh.row, &sh.tile);
    tc::fence_before();
    ptx::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = sh.tmem;
    const tc::Waits wait{&sh.gave_up};
    ptx::launch_dependents();
    Walk walk(p, sh, pair, pairs);
    Segment s;

    if (!kPaged && (warp == 5 || warp == 8)) {
        // Selected slots, first product: slots 64 rank + 32 part.. of each
        // tile, all values; 16 bytes a lane, four rows at a time.
        const int part = warp == 8 ? 1 : 0, r = lane >> 3;
        const int at = rank * kHalf + 32 * part + lane;
        int n = 0;
        bool more = walk.next(s);
        int tile = s.first;
        int next_slot = more ? slot_of<false>(p, s.row, s.length, static_cast<int64_t>(tile) * kTile + at) : -1;
        while (more && !wait.over()) {
            const int slot = next_slot;
            // The next tile's slots are fetched while this one's copies wait.
            if (++tile == s.last) {
                more = walk.next(s);
                tile = s.first;
            }
            if (more) next_slot = slot_of<false>(p, s.row, s.length, static_cast<int64_t>(tile) * kTile + at);
            const uint8_t* from[8];
            uint32_t bytes = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int x = __shfl_sync(~0u, slot, 4 * q + r);
                bytes |= (x >= 0 ? 1u : 0u) << q;
                from[q] = static_cast<const uint8_t*>(p.cache) + max(x, 0) * (2 * p.slot_stride) + (lane & 7) * 16;
            }
            for (int g = 0; g < kKeyGroups; ++g) {
                if (n > 0) wait.warp(&sh.key_empty[g], (n - 1) & 1);
                const uint32_t to = keys + 3 * g * kKeyPiece + part * 4096 + r * 128;
                const uint32_t even = to + (((lane & 7) ^ r) << 4), odd = to + (((lane & 7) ^ r ^ 4) << 4);
#pragma unroll
                for (int q = 0; q < 8; ++q)
#pragma unroll
                    for (int c = 0; c < 3; ++c)
                        tc::copy16((q & 1 ? odd : even) + q * 512 + c * kKeyPiece, from[q] + 128 * (3 * g + c),
                                   ((bytes >> q) & 1) * 16);
                tc::copy16_arrive(&sh.key_landed[g]);
            }
            ++n;
            if (part == 0 && lane == 0) sh.copied = n;
        }
        tc::copy16_drain();
    } else if (!kPaged && (warp == 6 || warp == 9)) {
        // Selected slots, second product: slots 64 part.. of each tile,
        // values 256 rank...
        const int part = warp == 9 ? 1 : 0, r = lane >> 3;
        int n = 0;
        bool more = walk.next(s);
        int tile = s.first;
        const auto fetch = [&](int* slots) {
            for (int i = 0; i < 2; ++i)
                slots[i] = slot_of<false>(p, s.row, s.length, static_cast<int64_t>(tile) * kTile + kHalf * part + 32 * i + lane);
        };
        int next_slots[2];
        if (more) fetch(next_slots);
        while (more && !wait.over()) {
            const int slots[2] = {next_slots[0], next_slots[1]};
            if (++tile == s.last) {
                more = walk.next(s);
                tile = s.first;
            }
            if (more) fetch(next_slots);
            // One bit a slot that is seen.  Place n % 4 was last read for tile
            // n - 4, whose second product the copies of tile n - 2 waited for.
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t bits = __ballot_sync(~0u, slots[i] >= 0);
                if (lane == 0) sh.mask[n & 3][2 * part + i] = bits;
            }
            if (lane == 0) ptx::mbar_arrive(&sh.mask_full[n & 3]);
            for (int g = 0; g < 2; ++g) {
                if (n > 0) wait.warp(&sh.value_empty[g], (n - 1) & 1);
                const uint32_t to = values + 2 * g * kValuePiece + part * kKeyPiece + r * 128;
                const uint32_t even = to + (((lane & 7) ^ r) << 4), odd = to + (((lane & 7) ^ r ^ 4) << 4);
                const uint8_t* cache = static_cast<const uint8_t*>(p.cache) + 512 * rank + 256 * g + (lane & 7) * 16;
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int x = __shfl_sync(~0u, slots[q >> 3], (4 * q + r) & 31);
                    const uint8_t* from = cache + max(x, 0) * (2 * p.slot_stride);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tc::copy16((q & 1 ? odd : even) + q * 512 + c * kValuePiece, from + 128 * c, x >= 0 ? 16 : 0);
                }
                tc::copy16_arrive(&sh.value_landed[g]);
            }
            ++n;
        }
        tc::copy16_drain();
    } else if (kPaged && warp == 5) {
        // Pages, first product: slots 64 rank.. of each tile, all values.
        int n = 0;
        bool more = walk.next(s);
        int tile = s.first;
        const bool mine = lane * box_rows < kHalf;
        const auto fetch = [&]() {  // row of the cache at which box `lane` begins
            const int x = mine ? slot_of<true>(p, s.row, s.length,
                                               static_cast<int64_t>(tile) * kTile + rank * kHalf + lane * box_rows)
                               : -1;
            return x < 0 ? p.num_slots : x;
        };
        int next_box = more ? fetch() : 0;
        while (more && !wait.over()) {
            const int box = next_box;
            if (++tile == s.last) {
                more = walk.next(s);
                tile = s.first;
            }
            if (more) next_box = fetch();
            for (int g = 0; g < kKeyGroups; ++g) {
                if (n > 0) wait.warp(&sh.key_empty[g], (n - 1) & 1);
                if (lane == 0) ptx::mbar_arrive_expect_tx(&sh.key_landed[g], 3 * kKeyPiece);
                __syncwarp();
                if (mine)
                    for (int c = 3 * g; c < 3 * g + 3; ++c)
                        tc::load_2d(keys + c * kKeyPiece + lane * box_rows * 128, &maps.cache, 64 * c, box,
                                    &sh.key_landed[g]);
            }
            ++n;
            // The rows of the next tile come to L2 while this one's are used:
            // shared memory has room for one tile only.
            if (more && mine)
                for (int c = 0; c < kPieces; ++c) tc::prefetch_2d(&maps.cache, 64 * c, next_box);
        }
        if (n > 0 && wait.over())
            for (int g = 0; g < kKeyGroups; ++g) tc::Waits::drain(&sh.key_landed[g], (n - 1) & 1);
    } else if (kPaged && warp == 6) {
        // Pages, second product: all slots of each tile, values 256 rank...
        int n = 0;
        bool more = walk.next(s);
        int tile = s.first;
        const auto fetch = [&](int* slots) {  // slots lane, lane + 32, ..
            for (int i = 0; i < 4; ++i)
                slots[i] = slot_of<true>(p, s.row, s.length, static_cast<int64_t>(tile) * kTile + 32 * i + lane);
        };
        int next_slots[4];
        if (more) fetch(next_slots);
        while (more && !wait.over()) {
            const int slots[4] = {next_slots[0], next_slots[1], next_slots[2], next_slots[3]};
            if (++tile == s.last) {
                more = walk.next(s);
                tile = s.first;
            }
            if (more) fetch(next_slots);
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // as for selected slots
                const uint32_t bits = __ballot_sync(~0u, slots[i] >= 0);
                if (lane == 0) sh.mask[n & 3][i] = bits;
            }
            if (lane == 0) ptx::mbar_arrive(&sh.mask_full[n & 3]);
            // Box `lane` starts at position lane * box_rows of the tile.
            const int at = lane * box_rows;
            int box = -1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int x = __shfl_sync(~0u, slots[i], at & 31);
                if ((at >> 5) == i) box = x;
            }
            if (box < 0) box = p.num_slots;
            for (int g = 0; g < 2; ++g) {
                if (n > 0) wait.warp(&sh.value_empty[g], (n - 1) & 1);
                if (lane == 0) ptx::mbar_arrive_expect_tx(&sh.value_landed[g], 2 * kValuePiece);
                __syncwarp();
                if (at < kTile)
                    for (int c = 2 * g; c < 2 * g + 2; ++c)
                        tc::load_2d(values + c * kValuePiece + at * 128, &maps.cache, 256 * rank + 64 * c, box,
                                    &sh.value_landed[g]);
            }
            ++n;
        }
        if (n > 0 && wait.over())
            for (int g = 0; g < 2; ++g) tc::Waits::drain(&sh.value_landed[g], (n - 1) & 1);
    } else if (warp == kQueryWarp) {
        if (lane == 0 && rank == 0 && pair > 0) {
            const int tiles = tiles_of(length_of(p, walk.row)), all = p.queries * p.heads;
            const int64_t start = sh.begin - walk.first;  // of the group's tiles
            Join join = {};
            if (walk.left > 0 && walk.first > 0 && run_start(sh.total, pair - 1, pairs) <= start) {
                // Runs that begin before the group's end, and the one before this.
                const int64_t last = sh.total < pairs ? start + tiles - 1 : ((start + tiles) * pairs - 1) / sh.total;
                join.parts = static_cast<int32_t>(last) - pair + 2;
                join.rows = min(all - walk.group * kRows, kRows);
                join.at = static_cast<int64_t>(walk.row) * all + walk.group * kRows;
            }
            static_cast<Join*>(p.workspace)[pair] = join;
        }
        if (lane == 0) {
            const uint32_t full = ptx::map_rank(ptx::smem_addr(&sh.query_full), 0);
            for (int n = 0; walk.next(s); ++n) {
                if (n > 0) wait(&sh.query_empty, (n - 1) & 1);
                if (rank == 0) ptx::mbar_arrive_expect_tx(&sh.query_full, 2 * kQueryBytes);
                const int m = s.group * kRows + rank * kHalf;
                for (int c = 0; c < kPieces; ++c) {
                    if (whole_rows) {
                        tc::load_4d_pair(queries + c * kKeyPiece, &maps.q, 64 * c, m, 0, s.row, full);
                    } else {
                        for (int i = 0; i < kHalf; ++i)
                            tc::load_4d_pair(queries + c * kKeyPiece + i * 128, &maps.q, 64 * c, (m + i) % p.heads,
                                             (m + i) / p.heads, s.row, full);
                    }
                }
                if (*wait.gave_up) {
                    if (rank == 0) tc::Waits::drain(&sh.query_full, n & 1);
                    break;
                }
            }
        }
    } else if (!kPaged && warp == kPrefetchWarp) {
        // The rows of the tile after the one being copied come to L2 while
        // that one's are used: shared memory has room for one tile only.
        const int at = rank * kHalf + lane;
        int n = 0;
        uint32_t spins = 0;
        uint64_t since = 0;
        bool over = false;
        while (!over && walk.next(s))
            for (int tile = s.first; tile < s.last && !over; ++tile, ++n) {
                int slots[2];
                for (int i = 0; i < 2; ++i)
                    slots[i] = slot_of<false>(p, s.row, s.length, static_cast<int64_t>(tile) * kTile + at + 32 * i);
                // Once the copies of the tile before are under way; a tile
                // whose own copies are needs no more help.
                while (!over && __any_sync(~0u, sh.copied < n)) over = wait.idle(spins, since);
                spins = 0;
                if (__any_sync(~0u, sh.copied > n)) continue;
                for (int i = 0; i < 2; ++i)
                    if (slots[i] >= 0) {
                        const uint8_t* row = static_cast<const uint8_t*>(p.cache) + slots[i] * (2 * p.slot_stride);
                        for (int c = 0; c < kPieces; ++c) ptx::prefetch_l2(row + 128 * c);
                    }
            }
    } else if (warp == 7) {
        // Tells the first block of each group of pieces that landed here,
        // those of keys and of values as they come.
        const int64_t tiles = walk.left;
        int64_t keys_done = 0, values_done = 0;
        int kg = 0, vg = 0;
        bool more = walk.next(s);
        int tile = s.first;
        uint32_t spins = 0;
        uint64_t since = 0;
        while (more && (keys_done < tiles || values_done < tiles)) {
            if (keys_done < tiles &&
                __any_sync(~0u, ptx::mbar_test_wait(&sh.key_landed[kg], static_cast<uint32_t>(keys_done) & 1))) {
                tc::fence_async();
                __syncwarp();
                if (lane == 0) tc::arrive_cluster(ptx::map_rank(ptx::smem_addr(&sh.key_full[kg]), 0));
                if (++kg == kKeyGroups) {
                    kg = 0;
                    ++keys_done;
                }
                spins = 0;
            } else if (values_done < tiles &&
                       __any_sync(~0u, ptx::mbar_test_wait(&sh.value_landed[vg], static_cast<uint32_t>(values_done) & 1))) {
                const int left = s.length - tile * kTile;
                if (kPaged && left < kTile) {
                    // Rows past the sequence's end may hold anything, and a
                    // weight of zero would not hide a NaN.
                    for (int i = max(left, 0) * 16 + lane; i < kTile * 16; i += 32)
                        ptx::sts_u4(values + (2 * vg + ((i >> 3) & 1)) * kValuePiece + (i >> 4) * 128 + (i & 7) * 16,
                                    make_uint4(0, 0, 0, 0));
                }
                tc::fence_async();
                __syncwarp();
                if (lane == 0) tc::arrive_cluster(ptx::map_rank(ptx::smem_addr(&sh.value_full[vg]), 0));
                if (++vg == 2) {
                    vg = 0;
                    ++values_done;
                    if (++tile == s.last && values_done < tiles) {
                        walk.next(s);
                        tile = s.first;
                    }
                }
                spins = 0;
            } else {
                if (wait.idle(spins, since)) break;
            }
        }
    } else if (warp == 4) {
        if (rank == 0) {
            const uint32_t score_instr = tc::instruction(kBf16, kRows, kTile, negate, false);
            const uint32_t sum_instr = tc::instruction(kBf16, kRows, 256, false, true);
            const uint64_t query_at = tc::operand(queries), key_at = tc::operand(keys), weight_at = tc::operand(weights),
                           value_at = tc::operand(values, kValuePiece);
            // A third of the first product of tile `scored`, at most one ahead
            // of the second (there are two score tiles), or a half of the
            // second product of tile `summed`: whichever has its operands, so
            // that neither waits behind the other's copies.
            const auto ready = [](uint64_t* bar, int64_t n) {
                return __any_sync(~0u, ptx::mbar_test_wait(bar, static_cast<uint32_t>(n) & 1));
            };
            const int64_t tiles = walk.left;
            int64_t scored = 0, summed = 0;
            int kg = 0, vg = 0, tile = 0, segment = -1;
            bool first[2] = {};  // whether tiles n - 1 and n, by n mod 2, begin their segments
            uint32_t spins = 0;
            uint64_t since = 0;
            s.first = s.last = 0;
            while (summed < tiles) {
                if (summed < scored && (vg > 0 || ready(&sh.weight, summed)) && ready(&sh.value_full[vg], summed)) {
                    const bool add = !first[summed & 1];
                    tc::fence_after();
                    if (tc::elect()) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            tc::mma<2>(tmem + 128 * vg, weight_at + (k >> 2) * (kKeyPiece >> 4) + 2 * (k & 3),
                                       value_at + 2 * vg * (kValuePiece >> 4) + 128 * k, sum_instr, add || k > 0);
                        tc::commit_pair(&sh.value_empty[vg]);
                        if (vg == 1) tc::commit_pair(&sh.sum);
                    }
                    __syncwarp();
                    vg ^= 1;
                    if (vg == 0) ++summed;
                    spins = 0;
                    continue;
                }
                if (scored < tiles && scored - summed < 2) {
                    if (tile == s.last) {
                        walk.next(s);
                        tile = s.first;
                        ++segment;
                    }
                    if ((kg > 0 || tile > s.first || ready(&sh.query_full, segment)) && ready(&sh.key_full[kg], scored)) {
                        const uint32_t d = tmem + kScore + kHalf * (static_cast<uint32_t>(scored) & 1);
                        tc::fence_after();
                        if (tc::elect()) {
#pragma unroll
                            for (int k = 0; k < 12; ++k) {
                                const uint32_t at = (3 * kg + (k >> 2)) * (kKeyPiece >> 4) + 2 * (k & 3);
                                tc::mma<2>(d, query_at + at, key_at + at, score_instr, (kg | k) != 0);
                            }
                            tc::commit_pair(&sh.key_empty[kg]);
                            if (kg == kKeyGroups - 1) {
                                tc::commit_pair(&sh.score[scored & 1]);
                                if (tile == s.last - 1) tc::commit_pair(&sh.query_empty);
                            }
                        }
                        __syncwarp();
                        if (++kg == kKeyGroups) {
                            kg = 0;
                            first[scored & 1] = tile == s.first;
                            ++tile;
                            ++scored;
                        }
                        spins = 0;
                        continue;
                    }
                }
                if (wait.idle(spins, since)) break;
            }
            if (tc::elect()) {
                tc::commit<2>(&sh.end);
                tc::Waits::drain(&sh.end, 0);
            }
        }
    } else if (warp < 4) {
        const int r = threadIdx.x & 63, half = threadIdx.x >> 6;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp) << 21);
        const uint32_t weight_full = ptx::map_rank(ptx::smem_addr(&sh.weight), 0);
        const uint32_t weight_row = weights + half * kKeyPiece + r * 128;
        const int all = p.queries * p.heads, part_rows = min(all, kRows);
        int n = 0;
        while (walk.next(s)) {
            const int m_row = s.group * kRows + rank * kHalf + r;
            const int limit = s.length - (p.queries - 1 - min(m_row / p.heads, p.queries - 1));
            float m = -INFINITY, l = 0.f;
            for (int tile = s.first; tile < s.last; ++tile, ++n) {
                wait.warp(&sh.mask_full[n & 3], (n >> 2) & 1);
                wait.warp(&sh.score[n & 1], (n >> 1) & 1);
                tc::fence_after();
                uint32_t raw_s[kHalf];
                tc::load32(lanes + kScore + kHalf * (n & 1), raw_s);
                tc::load32(lanes + kScore + kHalf * (n & 1) + 32, raw_s + 32);
                uint64_t seen = *reinterpret_cast<const uint64_t*>(&sh.mask[n & 3][2 * half]);
                const int left = limit - tile * kTile - half * kHalf;  // of this thread's slots
                if (left < kHalf) seen &= left <= 0 ? 0ull : (~0ull >> (kHalf - left));
                tc::wait_load();
                float* x = reinterpret_cast<float*>(raw_s);
                if (__any_sync(~0u, seen != ~0ull)) {
                    const uint32_t lo = static_cast<uint32_t>(seen), hi = static_cast<uint32_t>(seen >> 32);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (!((lo >> i) & 1)) x[i] = -INFINITY;
                        if (!((hi >> i) & 1)) x[32 + i] = -INFINITY;
                    }
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < kHalf; ++i) top[i & 3] = fmaxf(top[i & 3], x[i]);
                float tile_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale_log2;
                // The other half of the slots is with thread t ^ 64.
                sh.exchange[n & 1][threadIdx.x] = tile_top;
                asm volatile("bar.sync 1, 128;" ::: "memory");
                tile_top = fmaxf(tile_top, sh.exchange[n & 1][threadIdx.x ^ 64]);
                const bool raise = tile_top > m + kLag || (m == -INFINITY && tile_top > m);
                const float next = raise ? tile_top : m;
                const float by = raise ? tc::exp2_approx(m - next) : 1.f;
                m = next;
                l *= by;
                const float shift = m == -INFINITY ? 0.f : -m;
                uint32_t w[32];
                float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float a = tc::exp2_approx(fmaf(x[2 * i], scale_log2, shift));
                    const float b = tc::exp2_approx(fmaf(x[2 * i + 1], scale_log2, shift));
                    add[(2 * i) & 3] += a;
                    add[(2 * i + 1) & 3] += b;
                    w[i] = tc::pack<kBf16>(a, b);
                }
                l += (add[0] + add[1]) + (add[2] + add[3]);
                // The weights' place and the sums are free once the second
                // product of the tile before is done.
                if (n > 0) {
                    wait.warp(&sh.sum, (n - 1) & 1);
                    tc::fence_after();
                }
                if (tile > s.first && __any_sync(~0u, raise)) {
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        uint32_t o[32];
                        tc::load32(lanes + 32 * c, o);
                        tc::wait_load();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
                        tc::store32(lanes + 32 * c, o);
                    }
                    tc::wait_store();
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    ptx::sts_u4(weight_row + ((i ^ (r & 7)) << 4),
                                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
                tc::fence_async();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::arrive_cluster(weight_full);
            }
            // The sums of both halves, then the values 256 half.. of the row.
            wait.warp(&sh.sum, (n - 1) & 1);
            tc::fence_after();
            sh.exchange[n & 1][threadIdx.x] = l;
            asm volatile("bar.sync 1, 128;" ::: "memory");
            l += sh.exchange[n & 1][threadIdx.x ^ 64];
            // exchange[n & 1] is written again by the next tile n.
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const bool whole = s.first == 0 && s.last == s.tiles;
            const int64_t at = static_cast<int64_t>(s.row) * all + m_row;
            const int r_part = m_row - s.group * kRows;
            float* part = whole ? nullptr : part_of(p, part_rows, 2 * pair + (s.first == 0 ? 1 : 0));
            if (!whole && half == 0 && m_row < all)
                reinterpret_cast<float2*>(part + static_cast<int64_t>(part_rows) * kLatent)[r_part] = make_float2(m, l);
            const float by = l == 0.f ? 0.f : 1.f / l;
            uint16_t* out = static_cast<uint16_t*>(p.out) + at * kLatent + 256 * half;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
                uint32_t o[32];
                tc::load32(lanes + 32 * c, o);
                tc::wait_load();
                if (m_row < all && whole) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float a = __uint_as_float(o[16 * i + 2 * k]) * by,
                                        b = __uint_as_float(o[16 * i + 2 * k + 1]) * by;
                            w[k] = l == 0.f ? 0u : tc::pack<kBf16>(a, b);
                        }
                        tc::store_v8(out + 32 * c + 16 * i, w);
                    }
                } else if (m_row < all) {
                    uint4* to = reinterpret_cast<uint4*>(part) + static_cast<int64_t>(64 * half + 8 * c) * part_rows + r_part;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        to[i * part_rows] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
                __syncwarp();
            }
            if (whole && p.lse && half == 0 && m_row < all)
                p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            tc::fence_before();
        }
    }
    __syncwarp();
    // Neither block ends, nor gives its tensor memory back, while products of
    // the pair or copies may still use it.
    ptx::cluster_sync();
    if (warp == 4) {
        tc::fence_after();
        tc::dealloc<2>(tmem, kColumns);
    }
    if (threadIdx.x == 0 && sh.gave_up) atomicOr(flags, TOPK_FLAG_TIMEOUT);
}

// Joins the rows that several pairs shared: block (i, j) those of pair i + 1's
// Join, 16 values of 32 rows by each warp, a row a lane.
constexpr int kJoinThreads = 128;

template <bool kBf16>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const LatentParams p) {
    const int pair = static_cast<int>(blockIdx.x) + 1;
    ptx::grid_dependency_wait();
    const Join join = static_cast<const Join*>(p.workspace)[pair];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = static_cast<int>(blockIdx.y >> 3) * 32 + lane;
    const int c0 = 4 * (static_cast<int>(blockIdx.y & 7) * (kJoinThreads / 32) + warp);  // float4 columns
    if (r >= join.rows || join.parts == 0) return;
    const int part_rows = min(p.queries * p.heads, kRows);
    const auto stats_of = [&](int i) {
        const float* part = part_of(p, part_rows, 2 * (pair - 1 + i) + (i == 0 ? 1 : 0));
        return reinterpret_cast<const float2*>(part + static_cast<int64_t>(part_rows) * kLatent)[r];
    };
    float m = -INFINITY;
#pragma unroll 8
    for (int i = 0; i < join.parts; ++i) m = fmaxf(m, stats_of(i).x);
    if (m == -INFINITY) m = 0.f;
    float l = 0.f, o[16] = {};
#pragma unroll 4
    for (int i = 0; i < join.parts; ++i) {
        const float2 stats = stats_of(i);
        const float4* from = reinterpret_cast<const float4*>(part_of(p, part_rows, 2 * (pair - 1 + i) + (i == 0 ? 1 : 0))) +
                             static_cast<int64_t>(c0) * part_rows + r;
        // A part that saw nothing has no sums.
        const float by = stats.y == 0.f ? 0.f : exp2f(stats.x - m);
        l += stats.y * by;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float4 x = from[c * part_rows];
            o[4 * c] += x.x * by;
            o[4 * c + 1] += x.y * by;
            o[4 * c + 2] += x.z * by;
            o[4 * c + 3] += x.w * by;
        }
    }
    const float by = l == 0.f ? 0.f : 1.f / l;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = tc::pack<kBf16>(o[2 * i] * by, o[2 * i + 1] * by);
    const int64_t at = join.at + r;
    tc::store_v8(static_cast<uint16_t*>(p.out) + at * kLatent + 4 * c0, w);
    if (p.lse && c0 == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

size_t latent_workspace_bytes(int32_t, int32_t queries, int32_t heads) {
    const int64_t all = static_cast<int64_t>(queries) * heads;
    return kJoinBytes + static_cast<size_t>(2 * kMaxPairs) * static_cast<size_t>(all < kRows ? all : kRows) *
                            (kLatent + 2) * sizeof(float);
}

topk_status_t launch_latent(const LatentParams& p, topk_dtype_t dtype, const AttendDevice& device, cudaStream_t stream) {
    const bool bf16 = dtype == TOPK_BF16;
    LatentMaps maps;
    // Query rows: one dimension of (query, head) where those have one stride,
    // copied 64 rows at a time; else one row at a time.
    const bool whole_rows = p.queries == 1 || p.heads == 1 || p.q_query_stride == p.heads * p.q_head_stride;
    const int64_t any = 2 * kWidth;  // stride of a dimension of one entry
    const int64_t all = static_cast<int64_t>(p.queries) * p.heads;
    const int64_t rows = whole_rows ? all : p.heads;
    const int64_t row_step = whole_rows && p.heads == 1 ? p.q_query_stride : p.q_head_stride;
    const int64_t q_dims[4] = {kWidth, rows, whole_rows ? 1 : p.queries, p.batch};
    const int64_t q_steps[3] = {rows > 1 ? 2 * row_step : any, whole_rows ? any : 2 * p.q_query_stride,
                                p.batch > 1 ? 2 * p.q_row_stride : any};
    CUresult r = encode_map(&maps.q, bf16, p.q, 4, q_dims, q_steps, 1, whole_rows ? kHalf : 1);
    const int64_t c_dims[2] = {kWidth, p.num_slots}, c_steps[1] = {2 * p.slot_stride};
    // Pages of 16 slots or more go through the copy engine.
    const bool paged = !p.indices && p.log2_page >= 4;
    const int box_rows = paged && p.log2_page < 6 ? 1 << p.log2_page : kHalf;
    if (r == CUDA_SUCCESS) r = encode_map(&maps.cache, bf16, p.cache, 2, c_dims, c_steps, 1, box_rows);
    if (r != CUDA_SUCCESS) return api_cuda_fail(cudaErrorInvalidValue, "latent attention tensor map");

    const auto kernel = paged ? (bf16 ? latent_kernel<true, true> : latent_kernel<false, true>)
                              : (bf16 ? latent_kernel<true, false> : latent_kernel<false, false>);
    static std::atomic<bool> prepared[4][AttendDevice::kMax];
    cudaError_t e = allow_shared(kernel, kSmem, prepared[2 * paged + bf16][device.index]);
    if (e != cudaSuccess) return api_cuda_fail(e, "latent attention shared memory");
    const int64_t groups = (all + kRows - 1) / kRows;
    const int64_t tiles = p.batch * groups * (p.max_len > kTile ? (p.max_len + int64_t{kTile} - 1) / kTile : 1);
    const int64_t most = device.sms / 2 < kMaxPairs ? device.sms / 2 : kMaxPairs;
    const int pairs = static_cast<int>(tiles < most ? tiles : most);
    const float scale_log2 = std::fmax(std::fabs(p.scale) * 1.4426950408889634f, FLT_MIN);
    kernel<<<2 * pairs, kThreads, kSmem, stream>>>(p, maps, device.flags, scale_log2, p.scale < 0.f, whole_rows,
                                                  box_rows);
    e = cudaGetLastError();
    if (e != cudaSuccess) return api_cuda_fail(e, "latent attention launch");
    if (pairs > 1) {
        // Placed while the first kernel runs.
        cudaLaunchAttribute attr = {};
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(pairs - 1), 8 * static_cast<unsigned>(((all < kRows ? all : kRows) + 31) / 32));
        cfg.blockDim = dim3(kJoinThreads);
        cfg.stream = stream;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, bf16 ? join_kernel<true> : join_kernel<false>, p);
        if (e != cudaSuccess) return api_cuda_fail(e, "latent attention join launch");
    }
    return TOPK_OK;
}

}  // namespace topkidx
