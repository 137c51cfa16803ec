// index_scores.cu -- topk_index_scores: weighted scores of the indexer's heads
// over its paged keys, on the tensor cores.
//
// Mathematics: I[i][t] = sum_h w[i][h] max(q[i][h].k[t], 0) over 128 values a
// head.  Products of two-byte values are exact; all sums are fp32.  With D =
// K Q^T, 128 keys by up to 256 (query, head) columns, each key is a lane of
// tensor memory: the sum over a query's heads stays in one thread, and a warp
// writes 32 neighbouring scores.  A key's 256 bytes are read once for up to 512
// columns.  One query of 64 heads takes 16 K operations on 260 bytes and is
// bound by memory, 16 of them together by the products.
//
// Work is cut in runs of equal cost, one block an SM: the host does not know the
// lengths.  A tile (128 keys by one chunk of a request's queries) costs one, the
// beginning of a chunk one more where it is one product and two where it is
// two.  Tiles are independent, so nothing is joined.  A chunk's queries stay in shared memory
// while its keys pass through a ring of three to five places, by tiled copies of
// a page (or 128 rows of it) each; tensor memory holds two or four tiles of
// scores, some of them read while another is computed.
//
// Heads are padded to a power of two of columns, 16 or more, by the copy
// engine, with zeros: the loops over a query's columns are unrolled (a loop with
// its ends tested at run time took 1.5 times as long), and a chunk holds a power
// of two of queries, so that the cost of a request's tiles under the causal
// limit has a closed form.  Other numbers of heads pay for the next power of two,
// and for the test that keeps a padding column's infinity out of the sum: 4096
// queries on 4096 to 8192 keys take 325 us with 24 heads and 167 with 32, 2048 on
// 2048 to 4096 213 with 100 and 155 with 128.  (Where keys are finite a caller may
// pad the heads with zeros, of queries and of weights.)
//
// Measured: 128 requests of 1024 to 32768 keys, 64 heads, 89.9 us, 6.3 TB/s (92 %
// of the measured copy rate); one of 1048576 keys 47.4 us, 5.8 TB/s; 4096 queries
// of 64 heads on 4096 to 8192 keys 280 us alone, 297 in a row, 1.40 to 1.49
// PFLOP/s (82 to 87 % of the sustained rate of a library product): products and
// sums wait for one another through two tiles of scores, and the tensor pipe is
// busy 60 % of the time.  (Products of 128 columns and four tiles: 347 us, bound
// by shared memory; 16 warps of sums: 288; a tile given back as soon as its last
// columns are in registers, or the next tile's columns asked for then: 299 and
// 327; chunks of one product with two places: 297; pairs of blocks with half of
// the queries each: 287.)  4 requests of 8192 keys take 5 us on the GPU, of which
// 1.7 pass until a block knows its run and 2.2 more until its queries are there.
//
// Warps: 0-3 and 4-7 every other unit of a tile's columns, 8 products, 9 keys, 10
// queries and weights.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "attend_internal.h"
#include "tc.cuh"
#include "tensor_map.h"

namespace topkidx {
namespace {

constexpr int kThreads = 352;
constexpr int kProductWarp = 8, kKeyWarp = 9, kQueryWarp = 10;
constexpr int kTile = 128;  // 2^7
constexpr int kStages = 5, kBuffers = 4;       // tiles of keys and of scores, at most
constexpr int kMasks = kStages + kBuffers + 1;  // tiles whose masks are kept: those copied ahead and scored, and one
constexpr int kColumns = 256, kAllColumns = 2 * kColumns;  // of one product; of the queries in shared memory
constexpr int kHalfKeys = kTile * 128;                     // 64 values of a tile's keys
constexpr int kKeyBytes = 2 * kHalfKeys, kQueryBytes = 2 * kAllColumns * 128, kWeightBytes = kAllColumns * 4;
constexpr int kTileBytes = kQueryBytes + 3 * kKeyBytes;  // queries and keys

struct Span {  // of a request
    int32_t from, n, length;
};
struct Shared {
    uint64_t query_full[2], query_empty[2], weight_full[2];  // (full: by place; in one place by product)
    uint64_t key_full[kStages], key_empty[kStages], mask_full[kMasks];
    uint64_t score_full[kBuffers], score_empty[kBuffers], end;
    int64_t total, begin;  // units of cost of the whole call; the first of this block's run
    union {
        int64_t scan[kThreads / 32];  // until the run is found
        uint32_t mask[kMasks][4];
    };
    int32_t row, chunk, unit;  // where the run begins
    Span span;                 // of that row
    uint32_t tmem, gave_up;
};
// The structure lies before or behind the tiles, in what their alignment leaves.
constexpr int kSlack = 1024;
static_assert(sizeof(Shared) <= kSlack / 2, "barriers fit on one side");
constexpr int kSmem = kTileBytes + kWeightBytes + kSlack;
static_assert(kSmem <= 232448, "shared memory of a block");

struct ScoreMaps {
    CUtensorMap q, cache;
};
// How the columns are laid out: per query, product, chunk.
struct Layout {
    int32_t padded;      // heads, a power of two
    int32_t log2_queries;  // of a chunk
    int32_t begin_cost;    // of a chunk, in tiles
    int32_t product_queries;
    int32_t places;      // chunks in shared memory: 2 of one product or 1 of two
    int32_t place_columns;  // of each
    int32_t stages;      // tiles of keys in shared memory
    int32_t buffers;     // tiles of scores in tensor memory
    int32_t box_rows;    // keys per copy
    uint32_t instruction;  // without N
};

// A request's queries and what its tiles are.  Runs are cut by cost: a chunk's
// tiles and begin_cost more, for the change of queries in shared memory.
struct Request : Span {
    __device__ __forceinline__ Request(const Span& x) : Span(x) {}
    __device__ __forceinline__ Request(const IndexScoresParams& p, int b) {
        length = min(max(p.seq_lens[b], 0), p.max_len);
        if (p.cu_q) {
            from = min(max(p.cu_q[b], 0), p.total_q);
            n = max(min(max(p.cu_q[b + 1], 0), p.total_q) - from, 0);
        } else {
            n = p.total_q / p.batch;
            from = b * n;
        }
    }
    __device__ __forceinline__ int chunks(const Layout& a) const {
        return (n + (1 << a.log2_queries) - 1) >> a.log2_queries;
    }
    __device__ __forceinline__ int tiles(const Layout& a, int chunk) const {
        // Positions that the chunk's last query sees.
        const int seen = max(length - n + min(n, (chunk + 1) << a.log2_queries), 0);
        return static_cast<int>((static_cast<uint32_t>(seen) + kTile - 1) / kTile);
    }
    __device__ __forceinline__ int cost(const Layout& a, int chunk) const {
        const int x = tiles(a, chunk);
        return x > 0 ? x + a.begin_cost : 0;
    }
    // Cost of the chunks before `chunk`: whole ones, each sees 2^log2 more
    // than the one before, and 2^log2 divides a tile.
    __device__ __forceinline__ int64_t before(const Layout& a, int chunk) const {
        const int log2 = a.log2_queries, step = 1 << log2;
        const int blind = n > length ? (n - length) >> log2 : 0;  // chunks that see nothing
        if (chunk <= blind) return 0;
        const int64_t at = static_cast<int64_t>(length) - n + step + kTile - 1 + (static_cast<int64_t>(blind) << log2);
        const int log2_tile = 7 - log2;  // chunks of a tile's length
        const auto sum = [&](int64_t x) {  // of i >> log2_tile over i < x
            const int64_t q = x >> log2_tile;
            return ((q * (q - 1) / 2) << log2_tile) + (x & ((1 << log2_tile) - 1)) * q;
        };
        const int64_t i = at >> log2, many = chunk - blind;
        return sum(i + many) - sum(i) + many * a.begin_cost;
    }
    __device__ __forceinline__ int64_t all(const Layout& a) const {
        const int c = chunks(a);
        return c > 0 ? before(a, c - 1) + cost(a, c - 1) : 0;
    }
};

// The run of one of n blocks: as even as can be.
__device__ __forceinline__ int64_t run_start(int64_t total, int n, int i) {
    if (total <= INT32_MAX) {  // (a division of 64 bits takes some 100 instructions)
        const int each = static_cast<int>(total) / n, more = static_cast<int>(total) % n;
        return static_cast<int64_t>(each) * i + min(i, more);
    }
    return total / n * i + min(static_cast<int64_t>(i), total % n);
}

// All threads: the cost of the call, and where this block's run begins.
__device__ void locate(const IndexScoresParams& p, const Layout& a, Shared& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int from = min(tid * per, p.batch), to = min(from + per, p.batch);
    int64_t mine = 0;
    for (int b = from; b < to; ++b) mine += Request(p, b).all(a);
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(~0u, upto, d);
        if (lane >= d) upto += x;
    }
    if (lane == 31) sh.scan[warp] = upto;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const int64_t x = sh.scan[w];
        if (w < warp) before += x;
        total += x;
    }
    before += upto - mine;
    const int64_t begin = run_start(total, static_cast<int>(gridDim.x), static_cast<int>(blockIdx.x));
    if (tid == 0) {
        sh.total = total;
        sh.begin = begin;
    }
    if (begin >= before && begin < before + mine) {
        int64_t at = begin - before;
        int b = from;
        while (true) {
            const int64_t n = Request(p, b).all(a);
            if (at < n) break;
            at -= n;
            ++b;
        }
        const Request r(p, b);
        int lo = 0, hi = r.chunks(a) - 1;  // the last chunk with before <= at
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (r.before(a, mid) <= at)
                lo = mid;
            else
                hi = mid - 1;
        }
        sh.row = b;
        sh.chunk = lo;
        sh.unit = static_cast<int>(at - r.before(a, lo));
        sh.span = r;
    }
    __syncthreads();
}

// A run's pieces: tiles [first, last) of one chunk.
struct Segment {
    int row, query, queries, first, last;
    int seen;  // positions that the chunk's first query sees (may be below 1)
    int length;
};
struct Walk {
    const IndexScoresParams& p;
    const Layout& a;
    int64_t left;
    int row, chunk, first;  // (first: in units of cost)
    Request r;              // of the row

    __device__ __forceinline__ Walk(const IndexScoresParams& p, const Layout& a, const Shared& sh)
        : p(p), a(a), row(sh.row), chunk(sh.chunk), first(sh.unit), r(sh.span) {
        left = run_start(sh.total, static_cast<int>(gridDim.x), static_cast<int>(blockIdx.x) + 1) - sh.begin;
    }
    __device__ __forceinline__ bool next(Segment& s) {
        while (left > 0 && row < p.batch) {
            const int chunks = r.chunks(a);
            while (chunk < chunks && left > 0) {
                const int cost = r.cost(a, chunk), at = chunk << a.log2_queries;
                const int past = static_cast<int>(min(static_cast<int64_t>(cost), first + left));
                s.first = max(first - a.begin_cost, 0);
                s.last = past - a.begin_cost;
                left -= past - first;
                first = 0;
                ++chunk;
                if (s.last <= s.first) continue;
                s.row = row;
                s.query = r.from + at;
                s.queries = min(r.n - at, 1 << a.log2_queries);
                s.seen = r.length - (r.n - 1 - at);
                s.length = r.length;
                return true;
            }
            chunk = 0;
            if (++row < p.batch && left > 0) r = Request(p, row);
        }
        return false;
    }
};

// Columns of scores that a thread takes at a time, while the next are on their way.
constexpr int kStep = 32;
__device__ __forceinline__ void load_step(uint32_t from, uint32_t* to) {
#pragma unroll
    for (int i = 0; i < kStep; i += 32) tc::load32(from + i, to + i);
}

// Waits for what load_step asked for; nothing of it is used before.
__device__ __forceinline__ void landed(uint32_t* x) {
    tc::wait_load();
#pragma unroll
    for (int i = 0; i < kStep; ++i) asm volatile("" : "+r"(x[i]));
}

// sum += w max(x, 0) over kCount columns from `at` on, with the weights in shared
// memory; pairs of floats in 64 bits.  kFull: every column is a head.  Else
// those from `heads` on are zeros, but for a key that holds infinities.
template <int kCount, bool kFull>
__device__ __forceinline__ void add_part(const uint32_t* x, int at, int heads, uint32_t w_at, uint64_t* sum) {
    const auto top = [&](int i) {
        return ptx::fmax_nan(kFull || at + i < heads ? __uint_as_float(x[i]) : 0.f, 0.f);
    };
#pragma unroll
    for (int i = 0; i < kCount; i += 4) {
        uint64_t w[2];
        tc::load_pairs(w_at + 4 * i, w);
        sum[0] = tc::fma2(tc::pair(top(i), top(i + 1)), w[0], sum[0]);
        sum[1] = tc::fma2(tc::pair(top(i + 2), top(i + 3)), w[1], sum[1]);
    }
}

// kHeads: columns of a query.
template <int kHeads, bool kFull>
__global__ void __launch_bounds__(kThreads, 1)
    index_scores_kernel(const IndexScoresParams p, const __grid_constant__ ScoreMaps maps, const Layout a, uint32_t* flags) {
    extern __shared__ uint8_t raw[];
    const uint32_t start = ptx::smem_addr(raw), base = (start + kSlack - 1u) & ~(kSlack - 1u);
    const int place_columns = a.place_columns, place_bytes = place_columns * 256;
    const uint32_t queries = base, keys = queries + a.places * place_bytes, weights = base + kTileBytes;
    Shared& sh = *reinterpret_cast<Shared*>(raw + (base - start >= sizeof(Shared) ? 0 : weights + kWeightBytes - start));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        sh.gave_up = p.wait.none;
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sh.query_full[i], 1);
            ptx::mbar_init(&sh.query_empty[i], 9);  // the products, and each warp that reads the weights
            ptx::mbar_init(&sh.weight_full[i], 1);
        }
        for (int i = 0; i < kBuffers; ++i) {
            ptx::mbar_init(&sh.score_full[i], 1);
            ptx::mbar_init(&sh.score_empty[i], 8);
        }
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(&sh.key_full[i], 1);
            ptx::mbar_init(&sh.key_empty[i], 1);
        }
        for (int i = 0; i < kMasks; ++i) ptx::mbar_init(&sh.mask_full[i], 1);
        ptx::mbar_init(&sh.end, 1);
        ptx::fence_mbarrier_init();
    }
    if (warp == kKeyWarp && lane < 2) tc::prefetch_map(lane == 0 ? &maps.q : &maps.cache);
    if (warp == kProductWarp) tc::alloc<1>(ptx::smem_addr(&sh.tmem), 2 * kColumns);
    ptx::grid_dependency_wait();
    tc::fence_before();
    locate(p, a, sh);
    tc::fence_after();
    ptx::launch_dependents();
    const uint32_t tmem = sh.tmem;
    const tc::Waits wait{&sh.gave_up, p.wait.ns};
    Walk walk(p, a, sh);
    Segment s = {};

    if (warp == kKeyWarp) {
        int n = 0;
        bool more = walk.next(s);
        int tile = s.first;
        int32_t page[4];  // of positions lane, lane + 32, .. of the next tile; -1 past the row's end
        const int in_page = (1 << p.log2_page) - 1;
        const auto fetch = [&]() {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t t = static_cast<int64_t>(tile) * kTile + 32 * i + lane;
                page[i] = more && t < s.length ? p.table[static_cast<int64_t>(s.row) * p.table_stride + (t >> p.log2_page)] : -1;
            }
        };
        fetch();
        int stage = 0, round = 0, kept = 0;  // the place of tile n, how often it was filled, the mask's place
        while (more) {
            int slot[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int offset = (tile * kTile + 32 * i + lane) & in_page;
                const int64_t x = (static_cast<int64_t>(page[i]) << p.log2_page) + offset;
                slot[i] = x >= 0 && x < p.num_slots ? static_cast<int>(x) : -1;
            }
            if (++tile == s.last) {
                more = walk.next(s);
                tile = s.first;
            }
            fetch();
            if (round > 0 && !wait.all(&sh.key_empty[stage], (round - 1) & 1)) break;
            // The mask's place was last read for tile n - kMasks; the copies of
            // tile n waited for the products of tile n - stages, and those for
            // the sums of the score tile `buffers` before.
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t bits = __ballot_sync(~0u, slot[i] >= 0);
                if (lane == 0) sh.mask[kept][i] = bits;
            }
            if (lane == 0) {
                ptx::mbar_arrive(&sh.mask_full[kept]);
                ptx::mbar_arrive_expect_tx(&sh.key_full[stage], kKeyBytes);
            }
            __syncwarp();
            // A slot outside the cache is copied as zeros.
            for (int first = 0; first < kTile; first += 32 * a.box_rows) {
                const int at = first + lane * a.box_rows;
                int box = -1;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int x = __shfl_sync(~0u, slot[i], at & 31);
                    if ((at >> 5) == i) box = x;
                }
                if (box < 0) box = p.num_slots;
                if (at < kTile) {
                    tc::load_2d(keys + stage * kKeyBytes + at * 128, &maps.cache, 0, box, &sh.key_full[stage]);
                    tc::load_2d(keys + stage * kKeyBytes + kHalfKeys + at * 128, &maps.cache, 64, box, &sh.key_full[stage]);
                }
            }
            ++n;
            if (++stage == a.stages) {
                stage = 0;
                ++round;
            }
            if (++kept == kMasks) kept = 0;
        }
        for (int i = 0; i < a.stages; ++i) {
            const int copied = (n + a.stages - 1 - i) / a.stages;  // to this place
            if (copied > 0) tc::Waits::drain(&sh.key_full[i], (copied - 1) & 1);
        }
    } else if (warp == kQueryWarp) {
        uint32_t seconds = 0;  // second products so far
        for (int n = 0; walk.next(s); ++n) {
            const int place = n % a.places, round = n / a.places;
            // The first product begins without the second's queries.
            const int firsts = min(s.queries, a.product_queries), rest = s.queries - firsts;
            // Weights come to registers, and queries to L2, while the place is still in use.
            float w[kAllColumns / 32];
#pragma unroll
            for (int k = 0; k < kAllColumns / 32; ++k) {
                const int i = 32 * k + lane, q = i / kHeads, h = i % kHeads;
                w[k] = q < s.queries && h < p.heads ? p.weights[(s.query + q) * p.weights_stride + h] : 0.f;
            }
            if (round > 0) {
                for (int i = lane; i < 2 * s.queries; i += 32)
                    tc::prefetch_3d(&maps.q, 64 * (i & 1), 0, s.query + (i >> 1));
                if (!wait.all(&sh.query_empty[place], (round - 1) & 1) || wait.over()) break;
            }
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(&sh.query_full[place], firsts * kHeads * 256);
                if (rest > 0) ptx::mbar_arrive_expect_tx(&sh.query_full[1], rest * kHeads * 256);
            }
            __syncwarp();
            for (int i = lane; i < 2 * s.queries; i += 32)
                tc::load_3d(queries + place * place_bytes + (i & 1) * (place_columns * 128) + (i >> 1) * (kHeads * 128), &maps.q,
                            64 * (i & 1), 0, s.query + (i >> 1), &sh.query_full[(i >> 1) < firsts ? place : 1]);
#pragma unroll
            for (int k = 0; k < kAllColumns / 32; ++k)
                if (32 * k + lane < place_columns)
                    ptx::sts_u32(weights + 4 * (place * place_columns + 32 * k + lane), __float_as_uint(w[k]));
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sh.weight_full[place]);
            bool landed = wait.all(&sh.query_full[place], round & 1);
            if (rest > 0) landed = wait.all(&sh.query_full[1], seconds & 1) && landed;
            if (!landed) {
                tc::Waits::drain(&sh.query_full[place], round & 1);
                if (rest > 0) tc::Waits::drain(&sh.query_full[1], seconds & 1);
                break;
            }
            if (rest > 0) ++seconds;
        }
    } else if (warp == kProductWarp) {
        const uint64_t key_at = tc::operand(keys), query_at = tc::operand(queries);
        const uint32_t buffer_columns = 2 * kColumns / a.buffers;
        int stage = 0, buffer = 0;
        uint32_t round = 0, use = 0, seconds = 0;  // how often the places were used; second products
        // Given up, nothing is issued or announced any more.
        bool on = true;
        for (int segment = 0; walk.next(s); ++segment) {
            const int place = segment % a.places;
            on = wait.all(&sh.query_full[place], (segment / a.places) & 1) && on;
            for (int tile = s.first; tile < s.last; ++tile) {
                on = wait.all(&sh.key_full[stage], round & 1) && on;
                for (int first = 0; first < s.queries; first += a.product_queries) {
                    if (first > 0 && tile == s.first) on = wait.all(&sh.query_full[1], seconds++ & 1) && on;
                    if (use > 0) on = wait.all(&sh.score_empty[buffer], (use - 1) & 1) && on;
                    tc::fence_after();
                    if (on && tc::elect()) {
                        const int columns = min(s.queries - first, a.product_queries) * kHeads;
                        const uint32_t instr = a.instruction | (static_cast<uint32_t>(columns >> 3) << 17);
                        const uint64_t k_at = key_at + stage * (kKeyBytes >> 4);
                        const uint64_t q_at = query_at + ((place * place_bytes + first * kHeads * 128) >> 4);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            tc::mma<1>(tmem + buffer_columns * buffer, k_at + (k >> 2) * (kHalfKeys >> 4) + 2 * (k & 3),
                                       q_at + (k >> 2) * (place_columns * 8) + 2 * (k & 3), instr, k > 0);
                        tc::commit<1>(&sh.score_full[buffer]);
                        if (first + a.product_queries >= s.queries) {
                            tc::commit<1>(&sh.key_empty[stage]);
                            if (tile == s.last - 1) tc::commit<1>(&sh.query_empty[place]);
                        }
                    }
                    __syncwarp();
                    if (++buffer == a.buffers) {
                        buffer = 0;
                        ++use;
                    }
                }
                if (++stage == a.stages) {
                    stage = 0;
                    ++round;
                }
            }
        }
        if (tc::elect()) {
            tc::commit<1>(&sh.end);
            tc::Waits::drain(&sh.end, 0);
        }
    } else {
        const int half = warp >> 2, r = threadIdx.x & 127;
        const uint32_t buffer_columns = 2 * kColumns / a.buffers;
        // A unit of columns: a query or more, an even number of steps.
        constexpr int kUnit = kHeads > 2 * kStep ? kHeads : 2 * kStep, kUnitQueries = kUnit / kHeads;
        constexpr int kPart = kHeads < kStep ? kHeads : kStep;  // columns of one query in a step
        int kept = 0, buffer = 0;
        uint32_t round = 0, use = 0;  // of the masks' and the scores' places
        // These warps go through all tiles, also after a wait has given up.
        for (int segment = 0; walk.next(s); ++segment) {
            const int place = segment % a.places;
            const uint32_t weights_at = weights + place * (place_columns * 4);
            wait.warp(&sh.weight_full[place], (segment / a.places) & 1);
            for (int tile = s.first; tile < s.last; ++tile) {
                for (int first = 0; first < s.queries; first += a.product_queries) {
                    const int at = buffer;
                    const uint32_t phase = use & 1;
                    if (++buffer == a.buffers) {
                        buffer = 0;
                        ++use;
                    }
                    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21) + buffer_columns * at;
                    wait.warp(&sh.mask_full[kept], round & 1);
                    wait.warp(&sh.score_full[at], phase);
                    tc::fence_after();
                    const bool there = (sh.mask[kept][r >> 5] >> (r & 31)) & 1;
                    const int t = tile * kTile + r, count = min(s.queries - first, a.product_queries);
                    float* out = p.scores + (s.query + first) * p.scores_stride + t;
                    const int seen = s.seen + first;  // positions that the first of them sees
                    uint32_t x[2][kStep];
                    const int begin = half * kUnitQueries;
                    if (begin < count) load_step(lanes + begin * kHeads, x[0]);
                    for (int q = begin; q < count; q += 2 * kUnitQueries) {
                        const uint32_t w_at = weights_at + 4 * (first + q) * kHeads;
                        uint64_t sum[2] = {};
#pragma unroll
                        for (int c = 0; c < kUnit; c += kStep) {
                            uint32_t* now = x[c / kStep & 1];
                            landed(now);
                            // (columns behind the last query's are in this half of tensor memory too)
                            if (c + kStep < kUnit)
                                load_step(lanes + q * kHeads + c + kStep, x[(c / kStep + 1) & 1]);
                            else if (q + 2 * kUnitQueries < count)
                                load_step(lanes + (q + 2 * kUnitQueries) * kHeads, x[(c / kStep + 1) & 1]);
#pragma unroll
                            for (int i = 0; i < kStep; i += kPart) {
                                add_part<kPart, kFull>(now + i, (c + i) % kHeads, p.heads, w_at + 4 * (c + i), sum);
                                if ((c + i + kPart) % kHeads != 0) continue;
                                const int j = q + (c + i) / kHeads;
                                const float2 a = tc::unpair(sum[0]), b = tc::unpair(sum[1]);
                                if (j < count && t < seen + j) out[j * p.scores_stride] = there ? (a.x + a.y) + (b.x + b.y) : -INFINITY;
                                sum[0] = sum[1] = 0;
                            }
                        }
                    }
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&sh.score_empty[at]);
                }
                if (++kept == kMasks) {
                    kept = 0;
                    ++round;
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sh.query_empty[place]);
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == kProductWarp) {
        tc::fence_after();
        tc::dealloc<1>(tmem, 2 * kColumns);
    }
    if (threadIdx.x == 0 && sh.gave_up) atomicOr(flags, TOPK_FLAG_TIMEOUT);
}

}  // namespace

topk_status_t launch_index_scores(const IndexScoresParams& p, topk_dtype_t dtype, const AttendDevice& device, cudaStream_t stream) {
    const bool bf16 = dtype == TOPK_BF16;
    Layout a = {};
    int log2_heads = 4;
    while ((1 << log2_heads) < p.heads) ++log2_heads;
    a.padded = 1 << log2_heads;
    // Requests of few queries each: chunks of as many, the next one's come
    // while this one's are used, and what room they leave holds more tiles of
    // keys and of scores (three and two of them: one request of 1M keys 48.9
    // us in place of 47.3, 128 ragged ones 92.9 in place of 89.9).  The mean
    // decides: the host does not know how queries are spread (255 requests of one
    // query and one of 256, 4096 keys: 50.0 us, as two calls 52.8; 63 and one of
    // 512, 8192 keys: 77.1 and 71.1).  Else each key is read for two products (for
    // one: 4096 queries 297 us in place of 281), and a chunk that begins costs two
    // tiles (2.8 us; with runs of equal tiles 8 pieces of prompts took 39.8 us in
    // place of 28.7).
    const int most = 8 - log2_heads;  // log2 of a product's queries
    int log2 = 0;
    while (log2 <= most && (int64_t{p.batch} << log2) < p.total_q) ++log2;
    // Little work in all: smaller chunks, until there are tiles for one and a
    // half rounds of blocks (300 queries of 24 heads on 500 to 800 keys 14.7 ->
    // 11.1 us, 100 of 4 heads on 4100 keys 11.5 -> 10.0; for two rounds the first
    // took 11.9, for four 13.4).
    const int64_t key_tiles = (p.max_len + int64_t{kTile} - 1) / kTile;
    const auto tiles_of = [&](int x) {  // at most
        return (((static_cast<int64_t>(p.total_q) + (1 << x) - 1) >> x) + (x > 0 ? p.batch : 0)) * key_tiles;
    };
    while (log2 > 0 && 2 * tiles_of(log2) < 3 * device.sms) --log2;
    const bool small = log2 <= most;
    a.log2_queries = log2;
    a.product_queries = 1 << (small ? log2 : most);
    a.places = small ? 2 : 1;
    a.place_columns = a.padded << a.log2_queries;
    a.begin_cost = small ? 1 : 2;
    a.buffers = a.product_queries * a.padded <= kColumns / 2 ? kBuffers : 2;
    a.stages = (kTileBytes - a.places * a.place_columns * 256) / kKeyBytes;
    if (a.stages > kStages) a.stages = kStages;
    a.box_rows = p.log2_page < 7 ? 1 << p.log2_page : kTile;
    a.instruction = tc::instruction(bf16, kTile, 0, false, false);

    ScoreMaps maps;
    const int64_t any = 2 * kIndex;  // stride of a dimension of one entry
    const int64_t q_dims[3] = {kIndex, p.heads, p.total_q};
    const int64_t q_steps[2] = {p.heads > 1 ? 2 * p.q_head_stride : any, p.total_q > 1 ? 2 * p.q_token_stride : any};
    CUresult r = encode_map(&maps.q, bf16, p.q, 3, q_dims, q_steps, 1, a.padded);
    const int64_t c_dims[2] = {kIndex, p.num_slots}, c_steps[1] = {2 * p.slot_stride};
    if (r == CUDA_SUCCESS) r = encode_map(&maps.cache, bf16, p.cache, 2, c_dims, c_steps, 1, a.box_rows);
    if (r != CUDA_SUCCESS) return api_cuda_fail(cudaErrorInvalidValue, "index scores tensor map");

    using Kernel = decltype(&index_scores_kernel<16, true>);
    static constexpr Kernel kernels[2][5] = {
        {index_scores_kernel<16, false>, index_scores_kernel<32, false>, index_scores_kernel<64, false>,
         index_scores_kernel<128, false>, index_scores_kernel<256, false>},
        {index_scores_kernel<16, true>, index_scores_kernel<32, true>, index_scores_kernel<64, true>,
         index_scores_kernel<128, true>, index_scores_kernel<256, true>}};
    const bool full = p.heads == a.padded;
    const Kernel kernel = kernels[full][log2_heads - 4];
    static std::atomic<bool> prepared[2][5][AttendDevice::kMax];
    cudaError_t e = allow_shared(kernel, kSmem, prepared[full][log2_heads - 4][device.index]);
    if (e != cudaSuccess) return api_cuda_fail(e, "index scores shared memory");
    const int64_t tiles = tiles_of(log2);
    const unsigned blocks = static_cast<unsigned>(tiles < device.sms ? tiles : device.sms);
    e = launch_early(kernel, dim3(blocks), kThreads, kSmem, stream, p, maps, a, device.flags);
    return e == cudaSuccess ? TOPK_OK : api_cuda_fail(e, "index scores launch");
}

}  // namespace topkidx
