// tensor_core.cuh -- the 5th-generation tensor cores' instructions that the
// library uses: tcgen05.mma over operands in shared memory with accumulators in
// tensor memory, mbarriers and untiled bulk copies.
//
// Every wait has a limit of time.  One that runs out raises the block's abort
// word, at which the other roles' waits end as well.
#pragma once

#include <cstdint>

namespace sar {
namespace tc {

__device__ __forceinline__ uint32_t shared_address(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void barrier_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool barrier_test(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// The same, with what other blocks of the cluster did before they arrived.
__device__ __forceinline__ bool barrier_test_cluster(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
// 16 bytes of a block's shared memory, at an address that place_in gave.
__device__ __forceinline__ float4 load_cluster(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
    return v;
}
// The same barrier, or place in shared memory, in block `rank` of the cluster.
__device__ __forceinline__ uint32_t place_in(uint32_t bar, uint32_t rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(bar), "r"(rank));
    return at;
}
__device__ __forceinline__ void barrier_arrive_cluster(uint32_t bar_of_block) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_of_block) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// The longest wait, in ns: a kernel of these takes milliseconds.
constexpr uint64_t kWaitLimit = 2000000000ull;

__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

// Waits for the phase; false where the limit ran out (and then in every role:
// `aborted` is the block's word in shared memory).  With `aborted` null the wait
// is for the caller's own copies only.
template <bool CLUSTER = false> __device__ __forceinline__ bool barrier_wait(uint32_t bar, uint32_t parity, volatile int* aborted) {
    const auto test = [=]() { return CLUSTER ? barrier_test_cluster(bar, parity) : barrier_test(bar, parity); };
    if (test()) return true;
    const uint64_t start = now_ns();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (test()) return true;
        if (aborted != nullptr && *aborted != 0) return false;
        if (now_ns() - start > kWaitLimit) {
            if (aborted != nullptr) *aborted = 1;
            return false;
        }
    }
}

// bytes: a multiple of 16, both addresses on 16-byte boundaries.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

// Writes of earlier kernels before the asynchronous reads that follow.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// All 32 lanes of one warp (of each of the two blocks of a PAIR).  512 columns are
// all of the SM's tensor memory.
template <int COLUMNS, bool PAIR> __device__ __forceinline__ void tmem_alloc(uint32_t* where) {
    if (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_address(where)), "n"(COLUMNS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_address(where)), "n"(COLUMNS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <int COLUMNS, bool PAIR> __device__ __forceinline__ void tmem_free(uint32_t base) {
    if (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "n"(COLUMNS));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "n"(COLUMNS));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Operands in shared memory, rows of 128 bytes in the 128-byte swizzle (16-byte
// piece p of row r at p ^ (r & 7)), in groups of 8 rows that start on 1024-byte
// boundaries.  Along k in the rows ("K-major"): `stride` is from one group to
// the next.  Along the matrix's own rows or columns ("MN-major", 64 of them in a
// 128-byte row, one k a row): `lead` is from 64 of them to the next 64 and
// `stride` from 8 k to the next 8.
__device__ __forceinline__ uint64_t operand(uint32_t address, uint32_t lead, uint32_t stride) {
    return static_cast<uint64_t>((address >> 4) & 0x3FFF) | static_cast<uint64_t>((lead >> 4) & 0x3FFF) << 16 |
           static_cast<uint64_t>((stride >> 4) & 0x3FFF) << 32 | 1ull << 46 | 2ull << 61;
}

// fp16 x fp16 into binary32: M rows of A by N of B, either of them MN-major.
__host__ __device__ constexpr uint32_t instruction_f16(int m, int n, bool mn_major_a, bool mn_major_b) {
    return 1u << 4 | (mn_major_a ? 1u << 15 : 0u) | (mn_major_b ? 1u << 16 : 0u) | static_cast<uint32_t>(n >> 3) << 17 |
           static_cast<uint32_t>(m >> 4) << 24;
}

// One thread (PAIR: of the block of even rank): accumulators (+)= A B over k = 16.
// A pair of blocks multiplies M rows, half of them from each one's shared memory,
// by N, half of them from each as well; each block's tensor memory gets its rows.
template <bool PAIR> __device__ __forceinline__ void mma_f16(uint32_t acc, uint64_t a, uint64_t b, uint32_t instruction, bool add) {
    if (PAIR)
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(acc),
            "l"(a), "l"(b), "r"(instruction), "r"(static_cast<uint32_t>(add))
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(acc),
            "l"(a), "l"(b), "r"(instruction), "r"(static_cast<uint32_t>(add))
            : "memory");
}

// Arrives on the barrier (PAIR: in both blocks) once all of this thread's products
// so far are done.
template <bool PAIR> __device__ __forceinline__ void mma_commit(uint32_t bar) {
    if (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// All four warps of a group of 128 threads: the registers of each thread from
// here on, out of those that the block was launched with.
template <int N> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// 32 columns of the warp's 32 lanes (warp w of four: lanes 32 w ..); they are there
// after tmem_wait.
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}
// Everything loaded so far; the registers pass through, so that no use comes before.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]),
                   "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

}  // namespace tc
}  // namespace sar
