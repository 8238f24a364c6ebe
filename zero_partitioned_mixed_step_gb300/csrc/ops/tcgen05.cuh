// Inline PTX of the tensor-core path: mbarriers with bounded waits, TMA
// copies, tensor memory and tcgen05 products.  CG is the number of CTAs that
// work on one tile (1, or a pair of neighbouring SMs).
#pragma once

#include <cstdint>

namespace zo {

__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

// True in one thread of a (whole) warp; the compiler then knows that the
// branch has a single thread and keeps the operands of copies and products in
// uniform registers.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The address of `addr` (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// A float of another CTA's shared memory (an address from map_to).
__device__ __forceinline__ float load_cluster(uint32_t addr)
{
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    return x;
}

// ------------------------------------------------------------------ mbarriers

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

// An arrival at a barrier of this CTA.
__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// An arrival by the one thread of a warp that passes lane 0, without a branch,
// at a barrier of this CTA or, with CG = 2, of the pair's first one (an address
// from map_to).  What it orders is tensor memory (by the tcgen05 fences), so
// CTA scope is enough: a release at cluster scope waits for the thread's other
// stores, which measured three times the whole product's time.
template <int CG>
__device__ __forceinline__ void bar_arrive_lane0(uint32_t bar, int lane)
{
    if (CG == 1)
        asm volatile("{ .reg .pred p; setp.eq.s32 p, %1, 0; @p mbarrier.arrive.shared::cta.b64 _, [%0]; }" ::"r"(bar),
                     "r"(lane) : "memory");
    else
        asm volatile("{ .reg .pred p; setp.eq.s32 p, %1, 0; @p mbarrier.arrive.shared::cluster.b64 _, [%0]; }" ::"r"(bar),
                     "r"(lane) : "memory");
}

// One poll, about 150 cycles where the phase is over.  Where it is not, the
// hardware suspends the thread meanwhile: a poll that fails takes 1.4 us (the
// first 4; measured on a barrier that nothing arrives at).
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;"
                 " selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

// The same, never suspended.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;"
                 " selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

// The registers of a warpgroup's threads, given to or taken from the block's others.
template <int N>
__device__ __forceinline__ void registers_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Polls before a wait gives up: 1.5 s of failing ones, where the longest wait
// that ends is for a few blocks of a tile, microseconds.
constexpr int kWaitLimit = 1 << 20;
// Polls for a copy or a product in flight once a role has given up: 24 ms.
constexpr int kDrainLimit = 1 << 14;

// Waits for a barrier's phase; false when the polls run out or another role of
// the CTA has given up (*gave_up, in shared memory).
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *gave_up)
{
    for (int i = 0; i < kWaitLimit; ++i) {
        if (bar_try(bar, parity))
            return true;
        if (*gave_up)
            return false;
    }
    *gave_up = 1;
    return false;
}

// The same for a whole warp, with one answer.
__device__ __forceinline__ bool bar_wait_warp(uint32_t bar, uint32_t parity, volatile int *gave_up)
{
    return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, gave_up));
}

// ------------------------------------------------------------------ TMA

// A box of a 2-D map into this CTA's shared memory, its bytes counted at
// `bar` (with CG = 2 a barrier of the pair's first CTA).
template <int CG>
__device__ __forceinline__ void tma_load(uint32_t dst, const void *map, int32_t x, int32_t y, uint32_t bar)
{
    if (CG == 1)
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%2, %3}], [%4];"
                     ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%2, %3}], [%4];"
                     ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}

__device__ __forceinline__ void tma_store(const void *map, int32_t x, int32_t y, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(map), "r"(x), "r"(y), "r"(src) : "memory");
}

__device__ __forceinline__ void tma_add(const void *map, int32_t x, int32_t y, uint32_t src)
{
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(map), "r"(x), "r"(y), "r"(src) : "memory");
}

// 4 bytes from global to shared memory without a register in between (zero where
// `there` is false: nothing is read then), in groups of this thread.
__device__ __forceinline__ void copy4(uint32_t dst, const float *src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// At most N of this thread's groups still read shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_shared()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ------------------------------------------------------------------ tensor memory and products

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t columns)
{
    if (CG == 1)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
                     "tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::"r"(dst), "r"(columns)
                     : "memory");
    else
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
                     "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(dst), "r"(columns)
                     : "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns)
{
    if (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory descriptor of a K-major tile of 128-byte rows, 128-byte
// swizzle, 8 rows (1024 bytes) to a swizzle atom.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction descriptor: fp32 accumulators, 8-bit A and B (0 E4M3, 1 E5M2), both K-major.
__host__ __device__ constexpr uint32_t f8_instr(int a, int b, int m, int n)
{
    return 1u << 4 | (uint32_t)a << 7 | (uint32_t)b << 10 | (uint32_t)(n >> 3) << 17 |
           (uint32_t)(m >> 4) << 24;
}

// D[tmem] (+)= A B^T over 32 bytes of k; one thread.
template <int CG>
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t instr, bool add)
{
    if (CG == 1)
        asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }"
                     ::"r"(d), "l"(a), "l"(b), "r"(instr), "r"((uint32_t)add) : "memory");
    else
        asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p; }"
                     ::"r"(d), "l"(a), "l"(b), "r"(instr), "r"((uint32_t)add) : "memory");
}

// An arrival at `bar` (in both CTAs of a pair) when this thread's products so far are done.
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    if (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
                     " [%0], %1;" ::"r"(bar), "h"((uint16_t)3) : "memory");
}

// 32 neighbouring columns of this thread's lane (the warp's 32 lanes together).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t r[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11,"
                 " %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29,"
                 " %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
                   "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
                   "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
                   "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
}

// The same for 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t r[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11,"
                 " %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
                   "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
}

// The loads so far are in their registers; their first uses are volatile too
// (scale_add), so none is moved ahead of this.
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// acc += part * s, not moved ahead of the wait for `part`
__device__ __forceinline__ void scale_add(float &acc, uint32_t part, float s)
{
    asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(acc) : "f"(__uint_as_float(part)), "f"(s));
}

__device__ __forceinline__ float2 mul2(float s, float a, float b)  // (s a, s b) in one instruction
{
    float2 r;
    asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %2}; mov.b64 y, {%3, %4}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z; }"
        : "=f"(r.x), "=f"(r.y) : "f"(s), "f"(a), "f"(b));
    return r;
}

// A barrier among `count` threads; true where any of them passes `x`.
__device__ __forceinline__ bool barrier_or(int id, int count, bool x)
{
    uint32_t r;
    asm volatile("{ .reg .pred p, q; setp.ne.b32 p, %1, 0; barrier.cta.red.or.pred q, %2, %3, p;"
                 " selp.u32 %0, 1, 0, q; }"
                 : "=r"(r) : "r"((uint32_t)x), "r"(id), "r"(count) : "memory");
    return r != 0;
}
__device__ __forceinline__ void barrier_of(int id, int count)
{
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

}  // namespace zo
