// tc.cuh -- thin inline-PTX wrappers for the 5th-generation tensor cores
// (tcgen05, tensor memory), tiled bulk copies and bounded waits.
//
// Shared-memory tiles are rows of 128 bytes (64 two-byte values) under the
// 128-byte swizzle: the 16-byte piece c of row r lies at piece c ^ (r & 7) of
// that row, and tiles start on 1024 bytes.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "attend_internal.h"
#include "ptx.cuh"

namespace topkidx {
namespace tc {

// ------------------------------------------------------------- descriptors
// kind::f16 instruction: D fp32; A and B bf16 or fp16.  b_cols: B is stored
// with its N index contiguous (a row of 128 bytes holds 64 columns of one k).
__host__ __device__ constexpr uint32_t instruction(bool bf16, int m, int n, bool negate_a, bool b_cols) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((negate_a ? 1u : 0u) << 13) |
           ((b_cols ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// Shared-memory operand under the 128-byte swizzle.  K contiguous: groups of
// eight rows are 1024 bytes apart, 16 values of k are 32 bytes further on.  N
// contiguous (b_cols): groups of eight k are 1024 bytes apart, the next 64
// columns `columns` bytes; 16 values of k are 2048 bytes further on.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t columns = 16) {
    return (static_cast<uint64_t>((addr & 0x3ffffu) >> 4)) | (static_cast<uint64_t>(columns >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

// ------------------------------------------------------------ tensor memory
template <int kGroup>
__device__ __forceinline__ void alloc(uint32_t smem_result, uint32_t columns) {
    if constexpr (kGroup == 1)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_result),
                     "r"(columns)
                     : "memory");
    else
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_result),
                     "r"(columns)
                     : "memory");
}
template <int kGroup>
__device__ __forceinline__ void dealloc(uint32_t addr, uint32_t columns) {
    if constexpr (kGroup == 1) {
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
    } else {
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
    }
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this warp's 32 lanes (one lane a thread).
__device__ __forceinline__ void load32(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void store32(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// One lane of a converged warp, always the same one.  Products issued under it
// keep their descriptors in uniform registers (32.9 cycles a product of 128 x
// 128 x 16 by a pair, 45.5 under `lane == 0`).
__device__ __forceinline__ bool elect() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// 8 columns, for where registers are few.
__device__ __forceinline__ void load8(uint32_t addr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
}
__device__ __forceinline__ void store8(uint32_t addr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// -------------------------------------------------------------- products
// D[tmem] (+)= A B; issued by one thread.
template <int kGroup>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t instr, bool add) {
    if constexpr (kGroup == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(instr), "r"(static_cast<uint32_t>(add))
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(instr), "r"(static_cast<uint32_t>(add))
            : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t instr, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(instr), "r"(static_cast<uint32_t>(add))
        : "memory");
}
// Arrives on `bar` once every product issued by this thread so far is done.
template <int kGroup>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if constexpr (kGroup == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         ptx::smem_addr(bar))
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         ptx::smem_addr(bar))
                     : "memory");
}
// The same on the barrier at this offset in both blocks of a pair.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            ptx::smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// Generic-proxy writes of shared memory before tensor-core reads of it.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ------------------------------------------------------------- tiled copies
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(ptx::smem_addr(bar))
        : "memory");
}
// The same tile to L2 only.
__device__ __forceinline__ void prefetch_2d(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(ptx::smem_addr(bar))
        : "memory");
}

// The same tile to L2 only.
__device__ __forceinline__ void prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

__device__ __forceinline__ void load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(ptx::smem_addr(bar))
        : "memory");
}
// 16 bytes, or zeros where `bytes` is 0 (then nothing is read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Arrives on `bar` (one of its expected arrivals) once this thread's copy16s so far have landed.
__device__ __forceinline__ void copy16_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(ptx::smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void copy16_drain() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Arrival on a barrier of either block of the cluster.  What it announces lies
// in this block's own shared memory and is read by this SM's tensor core, so
// the order that is needed is fence_async's, before the arrival; a release for
// the whole cluster would wait for every access in flight (1000 to 4300 cycles
// under load).
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// -------------------------------------------------------------- arithmetic
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Pairs of floats in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
// The same for pairs that stay in 64 bits, from shared memory two at a time.
__device__ __forceinline__ void load_pairs(uint32_t addr, uint64_t* v) {
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(v[0]), "=l"(v[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// The largest of three (NaNs are passed over).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// 32 bytes, a whole sector (32-byte aligned).
__device__ __forceinline__ void store_v8(void* to, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// Two floats to two-byte values, `lo` in the low half.
template <bool kBf16>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    if constexpr (kBf16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Softmax weights are 2^(x - m) for a running reference m that follows the
// largest x so far: set to kHead below it, and raised when a tile's largest
// passes that by more than kLag (a rise scales the sums so far).  So the
// largest weight is between 2^kHead and 2^(kHead + kLag).
// bf16 has the range of fp32.  fp16 is 2^-14 to 65504 (steps of 2^-24 below):
// with the largest at 2^7 to 2^15 a weight keeps its 11 bits down to 2^-21 of
// the largest and is off by at most 2^-32 of it below that (at 1 to 2^8: by
// 2^-25, and 2000 slots 26 bits below one in their first tile were lost).
constexpr float kLag = 8.f;
template <bool kBf16>
constexpr float kHead = kBf16 ? 0.f : 7.f;

// ------------------------------------------------------------ bounded waits
// A wait gives up after a limit (2 s unless the tuning says otherwise), sets
// the block's flag and says so; from then on every wait of the block whose
// phase is not complete does the same at once, and the block goes on to its
// end on whatever its buffers hold.  No barrier that counts the bytes of tiled
// copies is armed twice meanwhile: a warp that copies stops where its wait gave
// up and sees no room that was announced after one that did (each kernel says
// how), or waits for each of its copies before the next.  So every barrier has
// at most one phase in flight to drain before the block ends.
constexpr uint64_t kDrainNs = 2000000000ull;  // whatever the limit of a wait is

struct Waits {
    volatile uint32_t* gave_up;  // in shared memory
    uint64_t limit_ns;

    // Whether the phase is complete; false: given up.
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        return ptx::mbar_test_wait(bar, parity) || slow(bar, parity);
    }
    // By a whole warp, which goes on together.  Each lane has its own answer, so
    // none may leave a loop by it (a vote cost 4 % of a long prompt).
    __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity) const {
        const bool done = (*this)(bar, parity);
        __syncwarp();
        return done;
    }
    // The same with one answer for the warp.
    __device__ __forceinline__ bool all(uint64_t* bar, uint32_t parity) const {
        return __all_sync(~0u, (*this)(bar, parity));
    }
    // For a warp that polls several barriers: counts a poll in which none was
    // ready, looks at the clock and the flag now and then, and says whether to
    // give up.  `spins` is 0 after one that was.
    __device__ __forceinline__ bool idle(uint32_t& spins, uint64_t& since) const {
        if ((++spins & 255) != 0) return false;
        const uint64_t now = ptx::global_timer_ns();
        if (spins == 256) since = now;
        if (now - since >= limit_ns) *gave_up = 1u;
        __syncwarp();
        return over();
    }
    __device__ __forceinline__ bool over() const { return __any_sync(~0u, *gave_up != 0u); }
    __device__ __forceinline__ bool slow(uint64_t* bar, uint32_t parity) const {
        const uint64_t t0 = ptx::global_timer_ns();
        while (!*gave_up) {
            if (ptx::mbar_try_wait_sleep(bar, parity, 20000u)) return true;
            if (ptx::global_timer_ns() - t0 >= limit_ns) *gave_up = 1u;
        }
        return false;
    }
    // For copies or products that may still be in flight when a block ends.
    __device__ __forceinline__ static void drain(uint64_t* bar, uint32_t parity) {
        (void)ptx::mbar_wait_bounded(bar, parity, kDrainNs);
    }
};

}  // namespace tc
}  // namespace topkidx
