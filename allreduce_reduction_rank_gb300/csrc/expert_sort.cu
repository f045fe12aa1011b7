// expert_sort.cu -- the tokens' choices sorted by expert.
//
// A stable counting sort by one thread-block cluster.  Warp w of the cluster
// has the w-th run of consecutive slots.
//   1. It walks its run, 32 slots at a time: lanes with the same expert find
//      each other (match_any), so a slot's rank within the run is the run's
//      count so far plus the peers in lower lanes.  The rank is left in
//      position[]; the warp's counts per expert are in shared memory.
//   2. Per expert, the counts are summed up over the warps of a block, and
//      over the blocks through distributed shared memory; the segments'
//      starts are the running sum of the padded counts over the experts.
//   3. Each warp walks its run again: place = start + slots of the expert in
//      earlier runs + rank.
// Each place is written by exactly one thread and no atomics are used, so the
// order is that of the slots.
#include <atomic>

#include "sar_device.cuh"
#include "sar_internal.h"

namespace sar {
namespace {

constexpr int kMaxThreads = 1024, kMaxBlocks = 16, kUnroll = 4;

// Expert of a slot, -1 outside 0 .. experts - 1.
template <typename Id> __device__ __forceinline__ int expert_of(Id id, int experts) {
    return id >= 0 && id < experts ? static_cast<int>(id) : -1;
}

__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A word of block `rank`'s shared memory, at the address of `p` in this one's.
__device__ __forceinline__ int ld_cluster(const int* p, unsigned rank) {
    uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p)), far;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(at), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(far) : "memory");
    return v;
}

template <typename Id>
__global__ void __launch_bounds__(kMaxThreads) sort_kernel(SortArgs a) {
    extern __shared__ int smem[];
    const int warps = blockDim.x >> 5, E = a.experts;
    int* hist = smem;                                 // [warps][E]: counts, then first places
    int* total = hist + warps * E;                    // [E]: this block's counts
    int* start = total + E;                           // [E + 1]: the segments' starts
    int* filled = start + E + 1;                      // [E]: the ends of their slots
    int* carry = filled + E;                          // [32]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nb = gridDim.x, block = blockIdx.x;
    int* mine = hist + warp * E;
    for (int i = lane; i < E; i += 32) mine[i] = 0;
    __syncwarp();
    pdl_wait();

    const Id* ids = static_cast<const Id*>(a.ids);
    const uint32_t runs = static_cast<uint32_t>(warps) * nb;
    const uint32_t per = ((a.slots + runs - 1) / runs + 31) / 32 * 32;
    const uint64_t begin = static_cast<uint64_t>(per) * (static_cast<uint32_t>(block) * warps + warp);
    const uint64_t end = begin + per < a.slots ? begin + per : a.slots;
    const unsigned below = (1u << lane) - 1;
    for (uint64_t i0 = begin; i0 < end; i0 += 32 * kUnroll) {
        int e[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t i = i0 + 32 * u + lane;
            e[u] = i < end ? expert_of<Id>(ids[i], E) : -1;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t i = i0 + 32 * u + lane;
            const unsigned peers = __match_any_sync(0xFFFFFFFFu, e[u]);
            const int before = e[u] >= 0 ? mine[e[u]] : 0;
            __syncwarp();
            if (e[u] >= 0 && (peers & below) == 0) mine[e[u]] = before + __popc(peers);
            __syncwarp();
            if (i < end) a.position[i] = before + __popc(peers & below);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int sum = 0;
        for (int w = 0; w < warps; ++w) {
            const int c = hist[w * E + e];
            hist[w * E + e] = sum;
            sum += c;
        }
        total[e] = sum;
    }
    cluster_sync();
    // Experts in tiles of the block's threads: counts over the cluster, and the
    // running sum of the padded counts.
    int done = 0;
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        int count = 0, before = 0;
        if (e < E) {
            for (int b = 0; b < nb; ++b) {
                const int c = ld_cluster(total + e, b);
                if (b < block) before += c;
                count += c;
            }
        }
        const int padded = (count + a.align - 1) / a.align * a.align;
        int up = padded;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, up, d);
            if (lane >= d) up += v;
        }
        if (lane == 31) carry[warp] = up;
        __syncthreads();
        int base = done, all = 0;
        for (int w = 0; w < warps; ++w) {
            const int c = carry[w];
            if (w < warp) base += c;
            all += c;
        }
        done += all;
        if (e < E) {
            const int first = base + up - padded;
            start[e] = first;
            filled[e] = first + count;
            if (block == 0) {
                a.counts[e] = count;
                a.offsets[e] = first;
            }
            for (int w = 0; w < warps; ++w) hist[w * E + e] += first + before;
        }
        __syncthreads();
    }
    if (block == 0 && threadIdx.x == 0) a.offsets[E] = done;
    if (a.source != nullptr) {                        // places without a slot: padding, and past the segments
        for (int e = block * warps + warp; e < E; e += static_cast<int>(runs)) {
            const uint32_t last = static_cast<uint32_t>(e + 1 < E ? start[e + 1] : done);
            for (uint32_t p = filled[e] + lane; p < last && p < a.capacity; p += 32) a.source[p] = -1;
        }
        for (uint64_t p = static_cast<uint64_t>(done) + block * blockDim.x + threadIdx.x; p < a.capacity;
             p += nb * blockDim.x)
            a.source[p] = -1;
    }
    for (uint64_t i0 = begin; i0 < end; i0 += 32 * kUnroll) {
        int e[kUnroll], rank[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t i = i0 + 32 * u + lane;
            e[u] = i < end ? expert_of<Id>(ids[i], E) : -1;
            rank[u] = i < end ? a.position[i] : 0;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t i = i0 + 32 * u + lane;
            int place = e[u] >= 0 ? mine[e[u]] + rank[u] : -1;
            if (static_cast<uint32_t>(place) >= a.capacity) place = -1;
            if (i < end) a.position[i] = place;
            if (place >= 0 && a.source != nullptr) a.source[place] = static_cast<int>(i);
        }
    }
    cluster_sync();                                   // no block leaves while another reads its counts
}

size_t smem_bytes(int warps, int experts) {
    return (static_cast<size_t>(warps) * experts + 3 * experts + 1 + 32) * sizeof(int);
}

template <typename Id> cudaError_t sort(const SortArgs& a, cudaStream_t s) {
    // Clusters above 8 blocks and shared memory above 48 KiB are allowed
    // explicitly, once per device (only a successful call is remembered).
    constexpr int kMaxDev = 64;
    static std::atomic<bool> allowed[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
    if (!allowed[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(sort_kernel<Id>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(sort_kernel<Id>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(smem_bytes(kMaxThreads / 32, SAR_MAX_EXPERTS)));
        if (e != cudaSuccess) return e;
        allowed[dev].store(true, std::memory_order_release);
    }
    // Runs of about 64 slots a warp, then as many blocks as that takes.
    unsigned threads = 64, blocks = 1;
    while (threads < kMaxThreads && threads * 2u < a.slots) threads *= 2;
    while (blocks < kMaxBlocks && static_cast<size_t>(blocks) * kMaxThreads * 4 < a.slots) blocks *= 2;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem_bytes(static_cast<int>(threads / 32), a.experts);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sort_kernel<Id>, a);
}

}  // namespace

cudaError_t launch_expert_sort(int id_bytes, const SortArgs& a, cudaStream_t s) {
    return id_bytes == 8 ? sort<long long>(a, s) : sort<int>(a, s);
}

}  // namespace sar
