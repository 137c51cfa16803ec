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
// and walks their slots in tiles.  One sum of 128 x 512 in fp32 alone would
// fill an SM's tensor memory, and 128 queries with 128 latent rows its shared
// memory; the pair splits both: products are issued for two SMs at once
// (cta_group::2, M = 128), block r holding the rows 64 r.. of A, half of B and
// the sums of its own rows.  For the first product B is its half of the tile's
// slots (all 576 values, K contiguous), for the second the values 256 r.. of all
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
// Measured (with the join): 16 rows of 32768 to 131072 tokens, pages of 64, 128
// heads 292 to 308 us, 4.9 to 5.2 TB/s (73 to 76 % of the measured copy rate) and
// 1.18 to 1.25 PFLOP/s, by memory and products together at the power limit; 2048
// rows of up to 512 slots, 16 heads 238 to 250 us, 4.8 to 5.1 TB/s; 128 rows of
// 2048 slots, 128 heads 83 to 85 us, of which about 8 us pass before the first
// product and 11 in the join; one such row 14.2 to 15.3 us, four fifths of it
// waiting for memory in turn.
//
// Warps of each block: 0-3 softmax and results (thread t: row t & 63, half t >> 6
// of the tile's slots, values 256 (t >> 6).. of the sums), 4 products (first
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

constexpr int kRows = 128;  // (query, head) rows of a pair
constexpr int kHalfRows = 64;
constexpr int kThreads = 384;
constexpr int kQueryWarp = 10, kPrefetchWarp = 11;
constexpr int kMaxPairs = 80;
constexpr int kPieces = kWidth / 64;             // 9
constexpr int kQueryBytes = kPieces * kHalfRows * 128;
constexpr uint32_t kColumns = 512;
constexpr uint32_t kScore = 256;  // column of the two score tiles; the sums have 0..255

// A step is 128 slots (N = 128: 32.9 cycles a product, N = 64: 25.8).  Shared
// memory has one place for it, which is freed and filled in parts: the keys by
// thirds of the 576 values, the values by halves of the slots.
constexpr int kTile = 128;
constexpr int kHalf = kTile / 2;  // slots of each block in the first product, of each thread in the softmax
constexpr int kKeyGroups = 3, kGroupPieces = kPieces / kKeyGroups;
constexpr int kValueGroups = 2;
constexpr int kKeyPiece = kHalf * 128;     // a block's slots of 64 values
constexpr int kValuePiece = kTile * 128;   // all slots of 64 values
constexpr int kWeightPiece = kHalfRows * 128;  // 64 rows of 64 weights
constexpr int kKeyBytes = kPieces * kKeyPiece, kValueBytes = 4 * kValuePiece, kWeightBytes = 2 * kWeightPiece;

struct Shared {
    // landed: in this block; full: in both (used in the first block).
    uint64_t query_landed[2], query_full[2], query_empty[2];
    uint64_t key_landed[kKeyGroups], key_full[kKeyGroups], key_empty[kKeyGroups];
    uint64_t value_landed[kValueGroups], value_full[kValueGroups], value_empty[kValueGroups];
    uint64_t score[2], weight, sum, end;
    uint64_t mask_full[4];
    uint32_t mask[4][4];
    float exchange[2][kRows];
    uint32_t tmem, gave_up;
    volatile int32_t copied;  // tiles whose first copies are all under way
    int32_t total;            // tiles of the whole batch
    int32_t begin;            // first tile of this pair's run
    int32_t row, tile, length;  // where that lies: row of the batch, tile in the row, the row's length
    int32_t scan[kThreads / 32];
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
__device__ __forceinline__ int tiles_of(int length) {
    return max(static_cast<int>((static_cast<uint32_t>(length) + kTile - 1) / kTile), 1);
}
__device__ __forceinline__ int groups_of(const LatentParams& p) { return (p.queries * p.heads + kRows - 1) / kRows; }

// The runs of n pairs over all tiles (both below 2^31), as even as can be: the
// first `more` pairs have one tile more than the others.  With fewer tiles than
// pairs the last pairs, past `used`, have none.
struct Runs {
    int each, more, used;
    __device__ __forceinline__ Runs(int total, int n) {
        used = min(n, total);
        each = total / used;
        more = total % used;
    }
    __device__ __forceinline__ int start(int i) const { return each * min(i, used) + min(i, more); }
    __device__ __forceinline__ int count(int i) const { return i < used ? each + (i < more ? 1 : 0) : 0; }
    // The pair whose run has a tile.
    __device__ __forceinline__ int of(int tile) const {
        const int head = more * (each + 1);
        return tile < head ? tile / (each + 1) : more + (tile - head) / each;
    }
};

// All threads of a block: the tiles of the whole batch, and where the run of
// `pair` begins (for a pair without one: at the last tile).
__device__ void locate(const LatentParams& p, int pair, int pairs, Shared& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int groups = groups_of(p);
    if (!p.seq_lens) {
        if (tid == 0) {
            const int each = tiles_of(p.max_len) * groups, total = each * p.batch;
            const int begin = Runs(total, pairs).start(pair), at = min(begin, total - 1);
            sh.total = total;
            sh.begin = begin;
            sh.row = at / each;
            sh.tile = at % each;
            sh.length = p.max_len;
        }
        __syncthreads();
        return;
    }
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int from = min(tid * per, p.batch), to = min(from + per, p.batch);
    int mine = 0;
#pragma unroll 4
    for (int b = from; b < to; ++b) mine += tiles_of(length_of(p, b));
    mine *= groups;
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(~0u, upto, d);
        if (lane >= d) upto += x;
    }
    if (lane == 31) sh.scan[warp] = upto;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const int x = sh.scan[w];
        if (w < warp) before += x;
        total += x;
    }
    before += upto - mine;
    const int begin = Runs(total, pairs).start(pair), tile = min(begin, total - 1);
    if (tile >= before && tile < before + mine) {
        int at = before, b = from, length = 0;
        while (true) {
            length = length_of(p, b);
            const int n = tiles_of(length) * groups;
            if (tile < at + n) break;
            at += n;
            ++b;
        }
        sh.total = total;
        sh.begin = begin;
        sh.row = b;
        sh.tile = tile - at;
        sh.length = length;
    }
    __syncthreads();
}

// A run's pieces: tiles [first, last) of one group of 128 rows.
struct Segment {
    int row, group, first, last, tiles, length;
};
struct Walk {
    const LatentParams& p;
    int left, row, group, first, groups, length;

    __device__ __forceinline__ Walk(const LatentParams& p, const Shared& sh, int pair, int pairs)
        : p(p), left(Runs(sh.total, pairs).count(pair)), row(sh.row), groups(groups_of(p)), length(sh.length) {
        const int tiles = tiles_of(length);
        group = sh.tile / tiles;
        first = sh.tile - group * tiles;
    }
    __device__ __forceinline__ bool next(Segment& s) {
        if (left <= 0) return false;
        s.row = row;
        s.group = group;
        s.length = length;
        s.tiles = tiles_of(length);
        s.first = first;
        s.last = min(s.tiles, first + left);
        left -= s.last - s.first;
        first = 0;
        if (++group == groups) {
            group = 0;
            ++row;
            if (left > 0) length = length_of(p, row);
        }
        return true;
    }
};

// A position's slot on its way: the index or the page as it is loaded (-1 past
// the row's end), looked at only when the slot is needed, so that the load's
// latency passes behind other work.
template <bool kPaged>
struct Slot {
    int32_t value, offset;

    __device__ __forceinline__ void fetch(const LatentParams& p, int row, int length, int64_t at) {
        value = -1;
        offset = 0;
        if (at >= length) return;
        if (!kPaged && p.indices) {
            value = p.indices[static_cast<int64_t>(row) * p.indices_stride + at];
        } else {
            const int pos = static_cast<int>(at);
            value = p.table[static_cast<int64_t>(row) * p.table_stride + (pos >> p.log2_page)];
            offset = pos & ((1 << p.log2_page) - 1);
        }
    }
    // The slot, -1 where it is not seen.
    __device__ __forceinline__ int get(const LatentParams& p) const {
        if (!kPaged && p.indices) return value >= 0 && value < p.num_slots ? value : -1;
        const int64_t s = (static_cast<int64_t>(value) << p.log2_page) + offset;
        return s >= 0 && s < p.num_slots ? static_cast<int>(s) : -1;
    }
};

// One slot a tile of a run, fetched two tiles ahead of its use: loads wait
// behind the copies that are under way.
struct SlotAhead {
    const LatentParams& p;
    Walk& walk;
    Segment& s;
    int at, tiles, tile;
    Slot<false> slot[2];
    bool more;

    __device__ __forceinline__ SlotAhead(const LatentParams& p, Walk& walk, Segment& s, int at)
        : p(p), walk(walk), s(s), at(at), tiles(walk.left), more(walk.next(s)) {
        tile = s.first;
        fetch(slot[0]);
        fetch(slot[1]);
    }
    __device__ __forceinline__ void fetch(Slot<false>& x) {
        x.fetch(p, s.row, more ? s.length : 0, static_cast<int64_t>(tile) * kTile + at);
        if (more && ++tile == s.last) {
            more = walk.next(s);
            tile = s.first;
        }
    }
    __device__ __forceinline__ int next() {
        const int x = slot[0].get(p);
        slot[0] = slot[1];
        fetch(slot[1]);
        return x;
    }
};

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

// Rows of a place: a multiple of 4, so that every place and its statistics
// start on 16 bytes.
__host__ __device__ __forceinline__ int part_rows_of(int64_t all) {
    return static_cast<int>(all < kRows ? (all + 3) / 4 * 4 : kRows);
}

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
    // Up to 64 rows: 32 a block, two places for queries, and half of the
    // softmax warps.
    const bool few = p.queries * p.heads <= kHalfRows;
    const int block_rows = few ? kHalfRows / 2 : kHalfRows, query_piece = block_rows * 128;

    if (threadIdx.x == 0) {
        sh.gave_up = p.wait.none;
        sh.copied = 0;
        for (int i = 0; i < kKeyGroups; ++i) {
            ptx::mbar_init(&sh.key_landed[i], kPaged ? 1 : 64);
            ptx::mbar_init(&sh.key_full[i], 2);
            ptx::mbar_init(&sh.key_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sh.value_landed[i], kPaged ? 1 : 64);
            ptx::mbar_init(&sh.value_full[i], 2);
            ptx::mbar_init(&sh.value_empty[i], 1);
            ptx::mbar_init(&sh.score[i], 1);
            ptx::mbar_init(&sh.query_landed[i], 1);
            ptx::mbar_init(&sh.query_full[i], 2);
            ptx::mbar_init(&sh.query_empty[i], 1);
        }
        ptx::mbar_init(&sh.weight, few ? 4 : 8);
        ptx::mbar_init(&sh.sum, 1);
        ptx::mbar_init(&sh.end, 1);
        for (int i = 0; i < 4; ++i) ptx::mbar_init(&sh.mask_full[i], kPaged ? 1 : 2);
        ptx::fence_mbarrier_init();
    }
    if (warp == 4) tc::alloc<2>(ptx::smem_addr(&sh.tmem), kColumns);
    ptx::grid_dependency_wait();
    locate(p, pair, pairs, sh);
    // Both blocks' barriers and tensor memory are ready from the wait on; the
    // first slots are fetched before it.
    tc::fence_before();
    ptx::cluster_arrive();
    ptx::launch_dependents();
    const auto pair_ready = [] {
        __syncwarp();
        ptx::cluster_wait();
        tc::fence_after();
    };
    const uint32_t tmem = sh.tmem;
    const tc::Waits wait{&sh.gave_up, p.wait.ns};
    Walk walk(p, sh, pair, pairs);
    Segment s = {};

    if (!kPaged && (warp == 5 || warp == 8)) {
        // Selected slots, first product: 32 of the block's 64 slots of each
        // tile, all values; 16 bytes a lane, four rows at a time.
        const int part = warp == 8 ? 1 : 0, r = lane >> 3;
        SlotAhead ahead(p, walk, s, rank * kHalf + 32 * part + lane);
        const int tiles = ahead.tiles;
        pair_ready();
        for (int n = 0; n < tiles && !wait.over(); ++n) {
            const int slot = ahead.next();
            const uint8_t* from[8];
            uint32_t seen = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int x = __shfl_sync(~0u, slot, 4 * q + r);
                seen |= (x >= 0 ? 1u : 0u) << q;
                from[q] = static_cast<const uint8_t*>(p.cache) + max(x, 0) * (2 * p.slot_stride) + (lane & 7) * 16;
            }
            for (int g = 0; g < kKeyGroups; ++g) {
                if (n > 0) wait.warp(&sh.key_empty[g], (n - 1) & 1);
                const uint32_t to = keys + kGroupPieces * g * kKeyPiece + part * 4096 + r * 128;
                const uint32_t even = to + (((lane & 7) ^ r) << 4), odd = to + (((lane & 7) ^ r ^ 4) << 4);
#pragma unroll
                for (int q = 0; q < 8; ++q)
#pragma unroll
                    for (int c = 0; c < kGroupPieces; ++c)
                        tc::copy16((q & 1 ? odd : even) + q * 512 + c * kKeyPiece, from[q] + 128 * (kGroupPieces * g + c),
                                   ((seen >> q) & 1) * 16);
                tc::copy16_arrive(&sh.key_landed[g]);
            }
            if (part == 0 && lane == 0) sh.copied = n + 1;
        }
        tc::copy16_drain();
    } else if (!kPaged && (warp == 6 || warp == 9)) {
        // Selected slots, second product: 32 of each half of the tile's
        // slots, values 256 rank...
        const int part = warp == 9 ? 1 : 0, r = lane >> 3;
        Walk walk2 = walk;
        Segment s2 = {};
        SlotAhead ahead[kValueGroups] = {SlotAhead(p, walk, s, 32 * part + lane), SlotAhead(p, walk2, s2, kHalf + 32 * part + lane)};
        const int tiles = ahead[0].tiles;
        pair_ready();
        for (int n = 0; n < tiles && !wait.over(); ++n) {
            const int slots[kValueGroups] = {ahead[0].next(), ahead[1].next()};
            // One bit a slot that is seen.  Place n % 4 was last read for tile
            // n - 4; the copies of tile n - 1 waited for the second product of
            // tile n - 2.
#pragma unroll
            for (int g = 0; g < kValueGroups; ++g) {
                const uint32_t bits = __ballot_sync(~0u, slots[g] >= 0);
                if (lane == 0) sh.mask[n & 3][2 * g + part] = bits;
            }
            if (lane == 0) ptx::mbar_arrive(&sh.mask_full[n & 3]);
            const uint8_t* cache = static_cast<const uint8_t*>(p.cache) + 512 * rank + (lane & 7) * 16;
#pragma unroll
            for (int g = 0; g < kValueGroups; ++g) {
                if (n > 0) wait.warp(&sh.value_empty[g], (n - 1) & 1);
                const uint32_t to = values + g * (kHalf * 128) + part * 4096 + r * 128;
                const uint32_t even = to + (((lane & 7) ^ r) << 4), odd = to + (((lane & 7) ^ r ^ 4) << 4);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int x = __shfl_sync(~0u, slots[g], 4 * q + r);
                    const uint8_t* from = cache + max(x, 0) * (2 * p.slot_stride);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        tc::copy16((q & 1 ? odd : even) + q * 512 + c * kValuePiece, from + 128 * c, x >= 0 ? 16 : 0);
                }
                tc::copy16_arrive(&sh.value_landed[g]);
            }
        }
        tc::copy16_drain();
    } else if (kPaged && warp == 5) {
        // Pages, first product: slots 64 rank.. of each tile, all values.
        int n = 0;
        bool more = walk.next(s);
        int tile = s.first;
        const bool mine = lane * box_rows < kHalf;
        Slot<true> next;  // at which box `lane` of the next tile begins
        const auto fetch = [&]() {
            next.fetch(p, s.row, more && mine ? s.length : 0, static_cast<int64_t>(tile) * kTile + rank * kHalf + lane * box_rows);
        };
        const auto row_of = [&]() {  // outside the cache: copied as zeros
            const int x = next.get(p);
            return x < 0 ? p.num_slots : x;
        };
        fetch();
        pair_ready();
        int stopped = kKeyGroups;  // the group that was not copied any more
        while (more && stopped == kKeyGroups) {
            const int box = row_of();
            if (++tile == s.last) {
                more = walk.next(s);
                tile = s.first;
            }
            fetch();
            for (int g = 0; g < kKeyGroups; ++g) {
                if (n > 0 && !wait.all(&sh.key_empty[g], (n - 1) & 1)) {
                    stopped = g;
                    break;
                }
                if (lane == 0) ptx::mbar_arrive_expect_tx(&sh.key_landed[g], kGroupPieces * kKeyPiece);
                __syncwarp();
                if (mine)
                    for (int c = kGroupPieces * g; c < kGroupPieces * (g + 1); ++c)
                        tc::load_2d(keys + c * kKeyPiece + lane * box_rows * 128, &maps.cache, 64 * c, box,
                                    &sh.key_landed[g]);
            }
            if (stopped < kKeyGroups) break;
            ++n;
            // The rows of the next tile come to L2 while this one's are used:
            // shared memory has room for one tile only.
            if (more && mine)
                for (int c = 0, row = row_of(); c < kPieces; ++c) tc::prefetch_2d(&maps.cache, 64 * c, row);
        }
        for (int g = 0; g < kKeyGroups; ++g) {
            const int copied = stopped < kKeyGroups && g < stopped ? n + 1 : n;
            if (copied > 0) tc::Waits::drain(&sh.key_landed[g], (copied - 1) & 1);
        }
    } else if (kPaged && warp == 6) {
        // Pages, second product: all slots of each tile, values 256 rank...
        int n = 0;
        bool more = walk.next(s);
        int tile = s.first;
        Slot<true> next[4];  // slots lane, lane + 32, .. of the next tile
        const auto fetch = [&]() {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                next[i].fetch(p, s.row, more ? s.length : 0, static_cast<int64_t>(tile) * kTile + 32 * i + lane);
        };
        fetch();
        pair_ready();
        int stopped = kValueGroups;
        while (more && stopped == kValueGroups) {
            const int slots[4] = {next[0].get(p), next[1].get(p), next[2].get(p), next[3].get(p)};
            if (++tile == s.last) {
                more = walk.next(s);
                tile = s.first;
            }
            fetch();
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
            for (int g = 0; g < kValueGroups; ++g) {
                if (n > 0 && !wait.all(&sh.value_empty[g], (n - 1) & 1)) {
                    stopped = g;
                    break;
                }
                if (lane == 0) ptx::mbar_arrive_expect_tx(&sh.value_landed[g], kValueBytes / kValueGroups);
                __syncwarp();
                if (at / kHalf == g)
                    for (int c = 0; c < 4; ++c)
                        tc::load_2d(values + c * kValuePiece + at * 128, &maps.cache, 256 * rank + 64 * c, box,
                                    &sh.value_landed[g]);
            }
            if (stopped < kValueGroups) break;
            ++n;
        }
        for (int g = 0; g < kValueGroups; ++g) {
            const int copied = stopped < kValueGroups && g < stopped ? n + 1 : n;
            if (copied > 0) tc::Waits::drain(&sh.value_landed[g], (copied - 1) & 1);
        }
    } else if (warp == kQueryWarp) {
        if (lane == 0 && rank == 0 && pair > 0) {
            const Runs runs(sh.total, pairs);
            const int tiles = tiles_of(walk.length), all = p.queries * p.heads;
            const int start = sh.begin - walk.first;  // of the group's tiles
            Join join = {};
            if (walk.left > 0 && walk.first > 0 && runs.start(pair - 1) <= start) {
                // The run before this, and those that begin before the group's end.
                join.parts = runs.of(start + tiles - 1) - pair + 2;
                join.rows = min(all - walk.group * kRows, kRows);
                join.at = static_cast<int64_t>(walk.row) * all + walk.group * kRows;
            }
            static_cast<Join*>(p.workspace)[pair] = join;
        }
        pair_ready();
        if (lane == 0) {
            const int places = few ? 2 : 1;
            for (int n = 0; walk.next(s); ++n) {
                const int place = n % places, round = n / places;
                const uint32_t to = queries + place * kPieces * query_piece;
                uint64_t* landed = &sh.query_landed[place];
                if (round > 0 && !wait(&sh.query_empty[place], (round - 1) & 1)) break;
                ptx::mbar_arrive_expect_tx(landed, kPieces * query_piece);
                const int m = s.group * kRows + rank * block_rows;
                for (int c = 0; c < kPieces; ++c) {
                    if (whole_rows) {
                        tc::load_4d(to + c * query_piece, &maps.q, 64 * c, m, 0, s.row, landed);
                    } else {
                        for (int i = 0; i < block_rows; ++i)
                            tc::load_4d(to + c * query_piece + i * 128, &maps.q, 64 * c, (m + i) % p.heads,
                                        (m + i) / p.heads, s.row, landed);
                    }
                }
                if (!wait(landed, round & 1)) {
                    tc::Waits::drain(landed, round & 1);
                    break;
                }
                tc::fence_async();
                tc::arrive_cluster(ptx::map_rank(ptx::smem_addr(&sh.query_full[place]), 0));
            }
        }
    } else if (!kPaged && warp == kPrefetchWarp) {
        // The rows of the tile after those being copied come to L2.
        const int at = rank * kHalf + lane;
        int n = 0;
        uint32_t spins = 0;
        uint64_t since = 0;
        bool over = false;
        pair_ready();
        while (!over && walk.next(s))
            for (int tile = s.first; tile < s.last && !over; ++tile, ++n) {
                Slot<false> slots[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    slots[i].fetch(p, s.row, s.length, static_cast<int64_t>(tile) * kTile + at + 32 * i);
                // Once the copies of the tile before are under way; a tile
                // whose own copies are needs no more help.
                while (!over && __any_sync(~0u, sh.copied < n)) over = wait.idle(spins, since);
                spins = 0;
                if (__any_sync(~0u, sh.copied > n)) continue;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int x = slots[i].get(p);
                    if (x < 0) continue;
                    const uint8_t* row = static_cast<const uint8_t*>(p.cache) + x * (2 * p.slot_stride);
                    for (int c = 0; c < kPieces; ++c) ptx::prefetch_l2(row + 128 * c);
                }
                __syncwarp();
            }
    } else if (warp == 7) {
        // Tells the first block of each group of pieces that landed here,
        // those of keys and of values as they come.
        const int tiles = walk.left;
        int keys_done = 0, values_done = 0, kg = 0, vg = 0;
        const bool more = walk.next(s);
        int tile = s.first;
        uint32_t spins = 0;
        uint64_t since = 0;
        pair_ready();
        const auto ready = [](uint64_t* bar, int n) {
            return __any_sync(~0u, ptx::mbar_test_wait(bar, static_cast<uint32_t>(n) & 1));
        };
        while (more && (keys_done < tiles || values_done < tiles)) {
            if (keys_done < tiles && ready(&sh.key_landed[kg], keys_done)) {
                tc::fence_async();
                __syncwarp();
                if (lane == 0) tc::arrive_cluster(ptx::map_rank(ptx::smem_addr(&sh.key_full[kg]), 0));
                if (++kg == kKeyGroups) {
                    kg = 0;
                    ++keys_done;
                }
                spins = 0;
            } else if (values_done < tiles && ready(&sh.value_landed[vg], values_done)) {
                const int left = s.length - tile * kTile - vg * kHalf;
                if (kPaged && left < kHalf) {
                    // Rows past the sequence's end may hold anything, and a
                    // weight of zero would not hide a NaN.
                    for (int i = max(left, 0) * 32 + lane; i < kHalf * 32; i += 32)
                        ptx::sts_u4(values + ((i >> 3) & 3) * kValuePiece + (vg * kHalf + (i >> 5)) * 128 + (i & 7) * 16,
                                    make_uint4(0, 0, 0, 0));
                }
                tc::fence_async();
                __syncwarp();
                if (lane == 0) tc::arrive_cluster(ptx::map_rank(ptx::smem_addr(&sh.value_full[vg]), 0));
                if (++vg == kValueGroups) {
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
        pair_ready();
        if (rank == 0) {
            const uint32_t score_instr = tc::instruction(kBf16, kRows, kTile, negate, false);
            const uint32_t sum_instr = tc::instruction(kBf16, kRows, 256, false, true);
            const uint64_t query_at = tc::operand(queries), key_at = tc::operand(keys), weight_at = tc::operand(weights),
                           value_at = tc::operand(values, kValuePiece);
            // The first product of tile n goes before the second of tile n - 1:
            // while that runs, the keys' last third of tile n + 1 lands and the
            // softmax of tile n is done (taken as their operands came instead,
            // pages were 2 to 4 % slower).
            const int tiles = walk.left;
            int n = 0, segment = 0;
            bool add = false;  // whether the sums of tile n - 1 are added to
            int left = 0;      // its slots, up to the row's end
            // Pages: given up, nothing is issued or announced any more, so that
            // the other block, which has a flag of its own, is told the truth.
            // (Copies of selected slots are waited for by those who made them,
            // whatever they were let loose by.)
            bool on = true;
            const auto sums = [&](int m) {
                on &= wait.warp(&sh.weight, static_cast<uint32_t>(m) & 1);
                tc::fence_after();
                for (int g = 0; g < kValueGroups; ++g) {
                    on &= wait.warp(&sh.value_full[g], static_cast<uint32_t>(m) & 1);
                    if (tc::elect() && (on || !kPaged)) {
                        // Weights past the row's end are zero: nothing to
                        // add (1662 rows of up to 41 slots: 76.6 -> 72.6 us;
                        // not copying those slots either: 73.7, and rows of
                        // 512 slots 2 % slower).
                        if (g * kHalf < left) {
#pragma unroll
                            for (int a = 0; a < 2; ++a)  // values 128 a.. of each block's 256
#pragma unroll
                                for (int k = 0; k < kHalf / 16; ++k)
                                    tc::mma<2>(tmem + 128 * a, weight_at + g * (kWeightPiece >> 4) + 2 * k,
                                               value_at + ((2 * a * kValuePiece + g * kHalf * 128) >> 4) + 128 * k,
                                               sum_instr, add || g > 0 || k > 0);
                        }
                        tc::commit_pair(&sh.value_empty[g]);
                        if (g == kValueGroups - 1) tc::commit_pair(&sh.sum);
                    }
                    __syncwarp();
                }
            };
            for (; walk.next(s); ++segment) {
                const int place = few ? segment & 1 : 0;
                const uint32_t round = static_cast<uint32_t>(few ? segment >> 1 : segment) & 1;
                const uint64_t q_at = query_at + place * (kPieces * query_piece >> 4);
                for (int tile = s.first; tile < s.last; ++tile, ++n) {
                    bool summed = n == 0;
                    if (tile == s.first) {
                        // Queries that are still on their way need not hold up
                        // the last sums of the segment before.
                        if (n > 0 && !__any_sync(~0u, ptx::mbar_test_wait(&sh.query_full[place], round))) {
                            sums(n - 1);
                            summed = true;
                        }
                        on &= wait.warp(&sh.query_full[place], round);
                    }
                    for (int g = 0; g < kKeyGroups; ++g) {
                        on &= wait.warp(&sh.key_full[g], static_cast<uint32_t>(n) & 1);
                        if (tc::elect() && (on || !kPaged)) {
#pragma unroll
                            for (int k = 0; k < 4 * kGroupPieces; ++k) {
                                const int c = kGroupPieces * g + (k >> 2);
                                tc::mma<2>(tmem + kScore + kHalf * (n & 1), q_at + c * (query_piece >> 4) + 2 * (k & 3),
                                           key_at + c * (kKeyPiece >> 4) + 2 * (k & 3), score_instr, (g | k) != 0);
                            }
                            tc::commit_pair(&sh.key_empty[g]);
                            if (g == kKeyGroups - 1) {
                                tc::commit_pair(&sh.score[n & 1]);
                                if (tile == s.last - 1) tc::commit_pair(&sh.query_empty[place]);
                            }
                        }
                        __syncwarp();
                    }
                    if (!summed) sums(n - 1);
                    add = tile > s.first;
                    left = s.length - tile * kTile;
                }
            }
            if (tiles > 0) sums(n - 1);
            if (tc::elect()) {
                tc::commit<2>(&sh.end);
                tc::Waits::drain(&sh.end, 0);
            }
        }
    } else if (warp < 4 && !(few && (warp & 1))) {
        const int r = threadIdx.x & 63, half = threadIdx.x >> 6;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp) << 21);
        const uint32_t weight_full = ptx::map_rank(ptx::smem_addr(&sh.weight), 0);
        const uint32_t weight_row = weights + half * kWeightPiece + r * 128;
        const int all = p.queries * p.heads, part_rows = part_rows_of(all);
        const int threads = few ? 64 : 128;
        const auto softmax_sync = [&] { asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory"); };
        int n = 0;
        // These warps wait for one another, so all of them go through all
        // tiles, also after one has given up.
        pair_ready();
        while (walk.next(s)) {
            const int m_row = s.group * kRows + rank * block_rows + r;
            const int limit = s.length - (p.queries - 1 - min(m_row / p.heads, p.queries - 1));
            float m = -INFINITY, l = 0.f;
            for (int tile = s.first; tile < s.last; ++tile, ++n) {
                wait.warp(&sh.mask_full[n & 3], (n >> 2) & 1);
                wait.warp(&sh.score[n & 1], (n >> 1) & 1);
                tc::fence_after();
                uint32_t raw_s[kHalf];
#pragma unroll
                for (int c = 0; c < kHalf / 32; ++c)
                    tc::load32(lanes + kScore + kHalf * (n & 1) + 32 * c, raw_s + 32 * c);
                uint32_t seen[kHalf / 32];
                bool all_seen = true;
                const int left = limit - tile * kTile - half * kHalf;  // of this thread's slots
#pragma unroll
                for (int c = 0; c < kHalf / 32; ++c) {
                    seen[c] = sh.mask[n & 3][half * (kHalf / 32) + c];
                    const int here = left - 32 * c;
                    if (here < 32) seen[c] &= here <= 0 ? 0u : (~0u >> (32 - here));
                    all_seen = all_seen && seen[c] == ~0u;
                }
                tc::wait_load();
                float* x = reinterpret_cast<float*>(raw_s);
                if (__any_sync(~0u, !all_seen)) {
#pragma unroll
                    for (int i = 0; i < kHalf; ++i)
                        if (!((seen[i >> 5] >> (i & 31)) & 1)) x[i] = -INFINITY;
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < kHalf; ++i) top[i & 3] = fmaxf(top[i & 3], x[i]);
                float tile_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale_log2;
                // The other half of the slots is with thread t ^ 64.
                sh.exchange[n & 1][threadIdx.x] = tile_top;
                softmax_sync();
                tile_top = fmaxf(tile_top, sh.exchange[n & 1][threadIdx.x ^ 64]);
                // (rows past the last see whatever is there)
                const bool raise = m_row < all && (tile_top > m + (tc::kHead<kBf16> + tc::kLag) || (m == -INFINITY && tile_top > m));
                const float next = raise ? tile_top - tc::kHead<kBf16> : m;
                const float by = raise ? tc::exp2_approx(m - next) : 1.f;
                m = next;
                l *= by;
                const float shift = m == -INFINITY ? 0.f : -m;
                uint32_t w[kHalf / 2];
                float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < kHalf / 2; ++i) {
                    const float a = tc::exp2_approx(fmaf(x[2 * i], scale_log2, shift));
                    const float b = tc::exp2_approx(fmaf(x[2 * i + 1], scale_log2, shift));
                    add[(2 * i) & 3] += a;
                    add[(2 * i + 1) & 3] += b;
                    w[i] = tc::pack<kBf16>(a, b);
                }
                l += (add[0] + add[1]) + (add[2] + add[3]);
                // The weights' place and the sums are free once the second
                // product of the tile before is done.
                if (n > 0) wait.warp(&sh.sum, (n - 1) & 1);
                if (tile > s.first && __any_sync(~0u, raise)) {
                    tc::fence_after();
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
            sh.exchange[n & 1][threadIdx.x] = l;
            softmax_sync();
            l += sh.exchange[n & 1][threadIdx.x ^ 64];
            // exchange[n & 1] is written again by the next tile n.
            softmax_sync();
            const bool whole = s.first == 0 && s.last == s.tiles;
            const int64_t at = static_cast<int64_t>(s.row) * all + m_row;
            const int r_part = m_row - s.group * kRows;
            float* part = whole ? nullptr : part_of(p, part_rows, 2 * pair + (s.first == 0 ? 1 : 0));
            if (!whole && half == 0 && m_row < all)
                reinterpret_cast<float2*>(part + static_cast<int64_t>(part_rows) * kLatent)[r_part] = make_float2(m, l);
            if (whole && p.lse && half == 0 && m_row < all)
                p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            const float by = l == 0.f ? 0.f : 1.f / l;
            uint16_t* out = static_cast<uint16_t*>(p.out) + at * kLatent + 256 * half;
            wait.warp(&sh.sum, (n - 1) & 1);
            tc::fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[64];
                tc::load32(lanes + 64 * c, o);
                tc::load32(lanes + 64 * c + 32, o + 32);
                tc::wait_load();
                if (m_row < all && whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float a = __uint_as_float(o[16 * i + 2 * k]) * by,
                                        b = __uint_as_float(o[16 * i + 2 * k + 1]) * by;
                            w[k] = l == 0.f ? 0u : tc::pack<kBf16>(a, b);
                        }
                        tc::store_v8(out + 64 * c + 16 * i, w);
                    }
                } else if (m_row < all) {
                    uint4* to = reinterpret_cast<uint4*>(part) + static_cast<int64_t>(64 * half + 16 * c) * part_rows + r_part;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        to[i * part_rows] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
                __syncwarp();
            }
            tc::fence_before();
        }
    } else {
        pair_ready();
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

// Joins the rows that several pairs shared.  Every block reads all pairs' Joins
// and takes its share of their units of 32 rows, a row a lane: with up to four
// parts a unit has 16 values a warp (whole 32-byte sectors of the result), with
// more of them four, so that a row of many parts has many threads; each has
// eight loads in flight.
constexpr int kJoinThreads = 256;
constexpr int kFewParts = 4;

// Values 4 c.. 4 (c + kColumns) of one row; kParts parts at a time.
template <bool kBf16, int kColumns, int kParts>
__device__ __forceinline__ void join_row(const LatentParams& p, const Join& join, int pair, int part_rows, int r, int c) {
    const auto part_at = [&](int i) { return part_of(p, part_rows, 2 * (pair - 1 + i) + (i == 0 ? 1 : 0)); };
    float m = -INFINITY, l = 0.f;
    float4 o[kColumns] = {};
    for (int i0 = 0; i0 < join.parts; i0 += kParts) {
        float2 stats[kParts];
        float4 x[kParts][kColumns];
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            stats[i] = make_float2(-INFINITY, 0.f);
            if (i0 + i < join.parts) {
                const float* part = part_at(i0 + i);
                stats[i] = reinterpret_cast<const float2*>(part + static_cast<int64_t>(part_rows) * kLatent)[r];
#pragma unroll
                for (int k = 0; k < kColumns; ++k)
                    x[i][k] = reinterpret_cast<const float4*>(part)[static_cast<int64_t>(c + k) * part_rows + r];
            }
        }
        // The maximum may rise: what is summed so far is scaled back.
        float top = m;
#pragma unroll
        for (int i = 0; i < kParts; ++i) top = fmaxf(top, stats[i].x);
        const float base = top == -INFINITY ? 0.f : top, back = exp2f(m - base);
        m = top;
        l *= back;
#pragma unroll
        for (int k = 0; k < kColumns; ++k) o[k] = make_float4(o[k].x * back, o[k].y * back, o[k].z * back, o[k].w * back);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            if (stats[i].y == 0.f) continue;  // a part that saw nothing
            const float by = exp2f(stats[i].x - base);
            l += stats[i].y * by;
#pragma unroll
            for (int k = 0; k < kColumns; ++k)
                o[k] = make_float4(o[k].x + x[i][k].x * by, o[k].y + x[i][k].y * by, o[k].z + x[i][k].z * by,
                                   o[k].w + x[i][k].w * by);
        }
    }
    const float by = l == 0.f ? 0.f : 1.f / l;
    const int64_t at = join.at + r;
    uint32_t w[2 * kColumns];
#pragma unroll
    for (int k = 0; k < kColumns; ++k) {
        w[2 * k] = tc::pack<kBf16>(o[k].x * by, o[k].y * by);
        w[2 * k + 1] = tc::pack<kBf16>(o[k].z * by, o[k].w * by);
    }
    uint16_t* out = static_cast<uint16_t*>(p.out) + at * kLatent + 4 * c;
    if constexpr (kColumns == 4)
        tc::store_v8(out, w);
    else
        *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
    if (p.lse && c == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <bool kBf16>
__global__ void __launch_bounds__(kJoinThreads, 2) join_kernel(const LatentParams p, int pairs) {
    __shared__ Join joins[kMaxPairs];
    __shared__ int upto[kMaxPairs];  // units of the Joins up to and with one
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (warp == 0) {
        constexpr int kRounds = (kMaxPairs + 31) / 32;
        Join mine[kRounds] = {};
#pragma unroll
        for (int k = 0; k < kRounds; ++k)
            if (32 * k + lane > 0 && 32 * k + lane < pairs) mine[k] = static_cast<const Join*>(p.workspace)[32 * k + lane];
        int before = 0;
#pragma unroll
        for (int k = 0; k < kRounds; ++k) {
            int units = mine[k].parts == 0 ? 0 : (mine[k].rows + 31) / 32 * (mine[k].parts <= kFewParts ? 4 : 16);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int x = __shfl_up_sync(~0u, units, d);
                if (lane >= d) units += x;
            }
            units += before;
            if (32 * k + lane < kMaxPairs) {
                joins[32 * k + lane] = mine[k];
                upto[32 * k + lane] = units;
            }
            before = __shfl_sync(~0u, units, 31);
        }
    }
    __syncthreads();
    const int part_rows = part_rows_of(p.queries * p.heads);
    for (int unit = static_cast<int>(blockIdx.x); unit < upto[kMaxPairs - 1]; unit += static_cast<int>(gridDim.x)) {
        int lo = 0, hi = kMaxPairs - 1;  // the first pair with upto > unit
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (upto[mid] > unit)
                hi = mid;
            else
                lo = mid + 1;
        }
        const Join join = joins[lo];
        const bool few = join.parts <= kFewParts;
        const int in_join = unit - (lo > 0 ? upto[lo - 1] : 0), columns = few ? 4 : 16;
        const int r = in_join / columns * 32 + lane, c = in_join % columns * 8 + warp;
        if (r >= join.rows) continue;
        if (few)
            join_row<kBf16, 4, 2>(p, join, lo, part_rows, r, 4 * c);
        else
            join_row<kBf16, 1, 8>(p, join, lo, part_rows, r, c);
    }
}

}  // namespace

size_t latent_workspace_bytes(int32_t, int32_t queries, int32_t heads) {
    const int64_t all = static_cast<int64_t>(queries) * heads;
    return kJoinBytes + static_cast<size_t>(2 * kMaxPairs) * static_cast<size_t>(part_rows_of(all)) *
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
    CUresult r = encode_map(&maps.q, bf16, p.q, 4, q_dims, q_steps, 1, !whole_rows ? 1 : all <= kHalfRows ? kHalfRows / 2 : kHalfRows);
    const int64_t c_dims[2] = {kWidth, p.num_slots}, c_steps[1] = {2 * p.slot_stride};
    // Pages of 16 slots or more go through the copy engine.
    const bool paged = !p.indices && p.log2_page >= 4;
    const int box_rows = paged && p.log2_page < 6 ? 1 << p.log2_page : 64;
    if (r == CUDA_SUCCESS) r = encode_map(&maps.cache, bf16, p.cache, 2, c_dims, c_steps, 1, box_rows);
    if (r != CUDA_SUCCESS) return api_cuda_fail(cudaErrorInvalidValue, "latent attention tensor map");

    const auto kernel = paged ? (bf16 ? latent_kernel<true, true> : latent_kernel<false, true>)
                              : (bf16 ? latent_kernel<true, false> : latent_kernel<false, false>);
    static std::atomic<bool> prepared[4][AttendDevice::kMax];
    cudaError_t e = allow_shared(kernel, kSmem, prepared[2 * paged + bf16][device.index]);
    if (e != cudaSuccess) return api_cuda_fail(e, "latent attention shared memory");
    const int64_t groups = (all + kRows - 1) / kRows;
    const int64_t tiles = p.batch * groups * (p.max_len > kTile ? (p.max_len + int64_t{kTile} - 1) / kTile : 1);
    if (tiles > INT32_MAX) return TOPK_EINVAL;
    const int64_t most = device.sms / 2 < kMaxPairs ? device.sms / 2 : kMaxPairs;
    const int pairs = static_cast<int>(tiles < most ? tiles : most);
    const float scale_log2 = std::fmax(std::fabs(p.scale) * 1.4426950408889634f, FLT_MIN);
    e = launch_early(kernel, dim3(2 * pairs), kThreads, kSmem, stream, p, maps, device.flags, scale_log2, p.scale < 0.f,
                     whole_rows, box_rows);
    if (e != cudaSuccess) return api_cuda_fail(e, "latent attention launch");
    if (pairs > 1) {
        const int units = (pairs - 1) * ((part_rows_of(all) + 31) / 32) * 16, blocks = 2 * device.sms;
        e = launch_early(bf16 ? join_kernel<true> : join_kernel<false>, dim3(units < blocks ? units : blocks), kJoinThreads,
                         0, stream, p, pairs);
        if (e != cudaSuccess) return api_cuda_fail(e, "latent attention join launch");
    }
    return TOPK_OK;
}

}  // namespace topkidx
