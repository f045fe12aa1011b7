// expert_sort.cu -- the tokens' choices sorted by expert.
//
// A stable counting sort.  A warp has a run of consecutive slots, 32 at a time:
// the lanes with its expert come from one ballot for each bit of the expert's
// number (four instructions a bit; match_any measured 100 cycles of an SM a
// warp), so a slot's rank within the run is the run's count so far plus its
// peers in lower lanes.  The places follow from the experts' counts in earlier
// runs of the block (shared memory), in earlier blocks, and the segments'
// starts, the running sum of the padded counts.
//
// Up to kTile slots one block does it all.  More slots take three launches over
// blocks of equal shares: count_kernel leaves each block's counts per expert at
// the start of the block's own part of position[] (a share has at least kTile
// slots, more than there can be experts), prefix_kernel sums them over the
// blocks in place and writes counts[], and place_kernel, whose blocks first
// take their counts out again, writes the places.  Each place is written by one
// thread and the only atomics add integers, so the order is that of the slots.
//
// Bound by latency: 65536 x 8 slots of 256 experts are 6 MB of traffic, 1 us of
// HBM time, and take 11.3 us (three launches of 2 us at the least; counts 3,
// prefixes 2.5, places 6); 32 x 8 slots take 1.9 us, one launch.  One cluster of
// 16 blocks for all of it took 57 us, tiles of 2048 and 6144 slots 15.4 and 15.5.
#include "sar_device.cuh"
#include "sar_internal.h"

namespace sar {
namespace {

constexpr unsigned kTile = 4096;                      // slots of one block, as many as 8191
constexpr int kMaxThreads = 1024, kRounds = 8;        // 32-slot rounds of a warp
static_assert(2 * kTile <= 1 << 13 && SAR_MAX_EXPERTS < 1 << 18, "an expert and a share's slot in one word");
static_assert(kTile >= SAR_MAX_EXPERTS, "a share's counts fit its part of position[]");

// Expert of a slot; `experts` for a dropped one.
template <typename Id> __device__ __forceinline__ int expert_of(Id id, int experts) {
    return id >= 0 && id < experts ? static_cast<int>(id) : experts;
}

// The blocks' shares of the slots: `per` each, the first `more` of them one more.
struct Shares {
    uint32_t blocks, per, more;
    __device__ __forceinline__ uint32_t start(uint32_t b) const { return per * b + (b < more ? b : more); }
};

template <typename Id> __global__ void __launch_bounds__(kMaxThreads) count_kernel(SortArgs a, Shares shares) {
    __shared__ int hist[SAR_MAX_EXPERTS];
    for (int e = threadIdx.x; e < a.experts; e += kMaxThreads) hist[e] = 0;
    pdl_wait();
    __syncthreads();
    const Id* ids = static_cast<const Id*>(a.ids);
    const uint32_t begin = shares.start(blockIdx.x), end = shares.start(blockIdx.x + 1);
    int e[kRounds];
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
        const uint32_t i = begin + u * kMaxThreads + threadIdx.x;
        e[u] = i < end ? expert_of<Id>(ids[i], a.experts) : a.experts;
    }
#pragma unroll
    for (int u = 0; u < kRounds; ++u)
        if (e[u] < a.experts) atomicAdd(&hist[e[u]], 1);
    __syncthreads();
    for (int k = threadIdx.x; k < a.experts; k += kMaxThreads) a.position[begin + k] = hist[k];
}

// 32 experts a block, a warp's lanes; the warps share the blocks' counts.
__global__ void __launch_bounds__(kMaxThreads) prefix_kernel(SortArgs a, Shares shares) {
    __shared__ int part[32][32];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    const uint32_t per = (shares.blocks + 31) / 32, b0 = per * warp, b1 = b0 + per < shares.blocks ? b0 + per : shares.blocks;
    // Four counts in flight at a time; the last four are still there for the
    // second walk, which is all of them up to 128 blocks.
    constexpr int kAhead = 4;
    int c[kAhead], sum = 0;
    auto fetch = [&](uint32_t b) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            c[i] = b + i < b1 && e < a.experts ? a.position[shares.start(b + i) + e] : 0;
    };
    for (uint32_t b = b0; b < b1; b += kAhead) {
        fetch(b);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) sum += c[i];
    }
    part[warp][lane] = sum;
    __syncthreads();
    if (warp == 0) {
        int all = 0;
#pragma unroll
        for (int w = 0; w < 32; ++w) {
            const int k = part[w][lane];
            part[w][lane] = all;
            all += k;
        }
        if (e < a.experts) a.counts[e] = all;
    }
    __syncthreads();
    int before = part[warp][lane];
    for (uint32_t b = b0; b < b1; b += kAhead) {
        if (per > kAhead) fetch(b);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (b + i < b1 && e < a.experts) a.position[shares.start(b + i) + e] = before;
            before += c[i];
        }
    }
}

// Places of one share of the slots; with kSingle the only one, which also
// counts.
template <typename Id, bool kSingle>
__global__ void __launch_bounds__(kMaxThreads) place_kernel(SortArgs a, Shares shares, int bits) {
    extern __shared__ int smem[];
    const int warps = blockDim.x >> 5, E = a.experts, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* hist = smem;                                 // [warps][E]: counts, then first places
    int* start = hist + warps * E;                    // [E]: the segments' starts
    int* filled = start + E;                          // [E]: the ends of their slots
    int* local = filled + E;                          // [E]: the segments' starts among this block's slots
    int* carry = local + E;                           // [2][32]
    int* sorted = carry + 64;                         // [slots of a share]: expert and slot, sorted
    int* mine = hist + warp * E;
    for (int i = lane; i < E; i += 32) mine[i] = 0;
    __syncwarp();
    pdl_wait();

    const Id* ids = static_cast<const Id*>(a.ids);
    const uint32_t begin = shares.start(blockIdx.x), end = shares.start(blockIdx.x + 1);
    const uint32_t rounds = (end - begin + blockDim.x - 1) / blockDim.x;
    const uint32_t first = begin + warp * rounds * 32 + lane;
    const unsigned below = (1u << lane) - 1;
    int e[kRounds], rank[kRounds];
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
        const uint32_t i = first + u * 32;
        e[u] = static_cast<uint32_t>(u) < rounds && i < end ? expert_of<Id>(ids[i], E) : E;
    }
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
        if (static_cast<uint32_t>(u) >= rounds) break;
        unsigned peers = 0xFFFFFFFFu;
        for (int b = 0; b < bits; ++b) {
            const bool one = (e[u] >> b) & 1;
            const unsigned with = __ballot_sync(0xFFFFFFFFu, one);
            peers &= one ? with : ~with;
        }
        const int before = e[u] < E ? mine[e[u]] : 0;
        __syncwarp();
        if (e[u] < E && (peers & below) == 0) mine[e[u]] = before + __popc(peers);
        __syncwarp();
        rank[u] = before + __popc(peers & below);
    }
    __syncthreads();
    // Experts in tiles of the block's threads.
    int done = 0, mine_done = 0;
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int x = e0 + threadIdx.x;
        int count = 0, before = 0, sum = 0;
        if (x < E) {
            for (int w0 = 0; w0 < warps; w0 += 8) {   // eight at a time in flight
                int c[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) c[w] = w0 + w < warps ? hist[(w0 + w) * E + x] : 0;
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    if (w0 + w < warps) hist[(w0 + w) * E + x] = sum;
                    sum += c[w];
                }
            }
            count = kSingle ? sum : a.counts[x];
            before = kSingle ? 0 : a.position[begin + x];
        }
        // Running sums over the experts: of the padded counts, and of the block's own.
        const int padded = (count + a.align - 1) / a.align * a.align;
        int up = padded, own = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, up, d), w = __shfl_up_sync(0xFFFFFFFFu, own, d);
            if (lane >= d) up += v, own += w;
        }
        if (lane == 31) carry[warp] = up, carry[32 + warp] = own;
        __syncthreads();
        const int c = lane < warps ? carry[lane] : 0, k = lane < warps ? carry[32 + lane] : 0;
        const int at = done + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? c : 0) + up - padded;
        const int here = mine_done + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? k : 0) + own - sum;
        done += __reduce_add_sync(0xFFFFFFFFu, c);
        mine_done += __reduce_add_sync(0xFFFFFFFFu, k);
        if (x < E) {
            start[x] = at + before;
            filled[x] = at + count;
            local[x] = here;
            if (blockIdx.x == 0) {
                if (kSingle) a.counts[x] = count;
                a.offsets[x] = at;
            }
        }
        __syncthreads();
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[E] = done;
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
        const uint32_t i = first + u * 32;
        if (static_cast<uint32_t>(u) >= rounds || i >= end) break;
        int place = -1;
        if (e[u] < E) {
            const int nth = mine[e[u]] + rank[u];     // of the expert's slots in this share
            place = start[e[u]] + nth;
            sorted[local[e[u]] + nth] = e[u] << 13 | static_cast<int>(i - begin);
        }
        a.position[i] = static_cast<uint32_t>(place) < a.capacity ? place : -1;
    }
    if (a.source != nullptr) {
        // In the order of the places, so that a warp's stores are runs and not 32
        // sectors each (65536 x 8 slots: 12.0 -> 11.3 us for the sort).
        __syncthreads();
        for (int n = threadIdx.x; n < mine_done; n += blockDim.x) {
            const int v = sorted[n], x = v >> 13;
            const uint32_t place = static_cast<uint32_t>(start[x] + n - local[x]);
            if (place < a.capacity) a.source[place] = static_cast<int>(begin + (v & 0x1FFF));
        }
    }
    if (a.source != nullptr) {                        // places without a slot: padding, and past the segments
        const unsigned runs = gridDim.x * warps;
        if (a.align > 1) {
            for (int x = blockIdx.x * warps + warp; x < E; x += static_cast<int>(runs)) {
                // up to the next segment's start
                const uint32_t from = filled[x];
                const uint32_t to = (from + a.align - 1) / a.align * a.align;
                for (uint32_t p = from + lane; p < to && p < a.capacity; p += 32) a.source[p] = -1;
            }
        }
        for (uint64_t p = static_cast<uint64_t>(done) + blockIdx.x * blockDim.x + threadIdx.x; p < a.capacity;
             p += static_cast<uint64_t>(gridDim.x) * blockDim.x)
            a.source[p] = -1;
    }
}

size_t smem_bytes(unsigned warps, int experts, uint32_t slots) {
    return (static_cast<size_t>(warps) * experts + 3 * static_cast<size_t>(experts) + 64 + slots) * sizeof(int);
}

template <typename Id, bool kSingle> cudaError_t place(const SortArgs& a, const Shares& shares, unsigned threads, cudaStream_t s) {
    // Shared memory above 48 KiB is allowed explicitly, once per device (only a
    // successful call is remembered).
    static std::atomic<bool> allowed[kDevices];
    const cudaError_t e = allow_smem(place_kernel<Id, kSingle>, smem_bytes(kMaxThreads / 32, SAR_MAX_EXPERTS, 2 * kTile), allowed);
    if (e != cudaSuccess) return e;
    int bits = 0;
    while (a.experts >> bits) ++bits;                 // of 0 .. experts
    return launch_kernel_smem(place_kernel<Id, kSingle>, dim3(shares.blocks), dim3(threads),
                              smem_bytes(threads / 32, a.experts, shares.per + 1), s, a, shares, bits);
}

template <typename Id> cudaError_t sort(const SortArgs& a, cudaStream_t s) {
    if (a.slots < 2 * kTile) {
        unsigned threads = 64;
        while (threads < kMaxThreads && threads < a.slots) threads *= 2;
        return place<Id, true>(a, {1, a.slots, 0}, threads, s);
    }
    const uint32_t blocks = a.slots / kTile;
    const Shares shares = {blocks, a.slots / blocks, a.slots % blocks};
    cudaError_t e = launch_kernel(count_kernel<Id>, dim3(blocks), dim3(kMaxThreads), s, a, shares);
    if (e != cudaSuccess) return e;
    e = launch_kernel(prefix_kernel, dim3((a.experts + 31) / 32), dim3(kMaxThreads), s, a, shares);
    if (e != cudaSuccess) return e;
    return place<Id, false>(a, shares, kMaxThreads, s);
}

}  // namespace

cudaError_t launch_expert_sort(int id_bytes, const SortArgs& a, cudaStream_t s) {
    return id_bytes == 8 ? sort<long long>(a, s) : sort<int>(a, s);
}

}  // namespace sar
