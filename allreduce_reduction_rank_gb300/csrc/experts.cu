// experts.cu -- tokens sorted by expert, their rows dispatched and combined.
//
// First form: one block sorts; one block per token (or segment's padding)
// moves rows element by element.
//
// The sort is a stable counting sort.  Warp w of the block has the w-th run of
// consecutive slots.  It counts its slots per expert, 32 at a time: lanes with
// the same expert find each other (match_any), the lowest adds their number.
// The exclusive sum of the counts over the warps, per expert, gives every warp
// its first place in each segment, and a second walk over the slots hands the
// places out in order.
#include "sar_device.cuh"
#include "sar_internal.h"

namespace sar {
namespace {

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;

__device__ __forceinline__ int expert_of(const void* ids, int id_bytes, size_t i, int experts) {
    const long long e = id_bytes == 8 ? static_cast<const long long*>(ids)[i]
                                      : static_cast<long long>(static_cast<const int*>(ids)[i]);
    return e >= 0 && e < experts ? static_cast<int>(e) : -1;
}

__global__ void __launch_bounds__(kSortThreads) sort_kernel(SortArgs a, int id_bytes) {
    extern __shared__ int hist[];                   // [kSortWarps][experts], then [experts + 1] offsets
    int* offs = hist + kSortWarps * a.experts;
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* mine = hist + warp * a.experts;
    for (int i = threadIdx.x; i < kSortWarps * a.experts; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    const size_t per = (static_cast<size_t>(a.slots) + kSortThreads - 1) / kSortThreads * 32;
    const size_t begin = per * warp, end = begin + per < a.slots ? begin + per : a.slots;
    for (size_t i0 = begin; i0 < end; i0 += 32) {
        const size_t i = i0 + lane;
        const int e = i < end ? expert_of(a.ids, id_bytes, i, a.experts) : -1;
        const unsigned peers = __match_any_sync(0xFFFFFFFFu, e);
        if (e >= 0 && lane == __ffs(peers) - 1) mine[e] += __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kSortThreads) {
        int sum = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = hist[w * a.experts + e];
            hist[w * a.experts + e] = sum;
            sum += c;
        }
        a.counts[e] = sum;
        offs[e + 1] = (sum + a.align - 1) / a.align * a.align;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        offs[0] = 0;
        for (int e = 0; e < a.experts; ++e) offs[e + 1] += offs[e];
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= a.experts; e += kSortThreads) a.offsets[e] = offs[e];
    if (a.source != nullptr) {
        for (uint32_t p = threadIdx.x; p < a.capacity; p += kSortThreads) a.source[p] = -1;
    }
    __syncthreads();
    for (size_t i0 = begin; i0 < end; i0 += 32) {
        const size_t i = i0 + lane;
        const int e = i < end ? expert_of(a.ids, id_bytes, i, a.experts) : -1;
        const unsigned peers = __match_any_sync(0xFFFFFFFFu, e);
        int place = -1;
        if (e >= 0) place = offs[e] + mine[e] + __popc(peers & ((1u << lane) - 1));
        __syncwarp();
        if (e >= 0 && lane == __ffs(peers) - 1) mine[e] += __popc(peers);
        __syncwarp();
        if (place >= 0 && static_cast<uint32_t>(place) >= a.capacity) place = -1;
        if (i < end) a.position[i] = place;
        if (place >= 0 && a.source != nullptr) a.source[place] = static_cast<int>(i);
    }
}

// Rows of the padding of segment e: offsets[e] + counts[e] .. offsets[e + 1] - 1,
// as far as they exist.
template <typename T> __device__ void clear_padding(const ExpertArgs& a, size_t e) {
    const long long first = static_cast<long long>(a.offsets[e]) + a.counts[e];
    const long long last = a.offsets[e + 1] < a.capacity ? a.offsets[e + 1] : static_cast<long long>(a.capacity);
    for (long long p = first; p < last; ++p)
        for (size_t c = threadIdx.x; c < a.cols; c += blockDim.x)
            static_cast<T*>(a.out)[static_cast<size_t>(p) * a.ldo + c] = T(0);
}

__device__ __forceinline__ bool kept(const ExpertArgs& a, int p) {
    return p >= 0 && static_cast<uint32_t>(p) < a.capacity;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(ExpertArgs a) {
    pdl_wait();
    const size_t n = a.tokens + (a.counts != nullptr ? a.experts : 0);
    for (size_t t = blockIdx.x; t < n; t += gridDim.x) {
        if (t >= a.tokens) {
            clear_padding<T>(a, t - a.tokens);
            continue;
        }
        for (size_t c = threadIdx.x; c < a.cols; c += kThreads) {
            const T v = static_cast<const T*>(a.tok)[t * a.ldt + c];
            for (int j = 0; j < a.topk; ++j) {
                const int p = a.position[t * a.topk + j];
                if (kept(a, p)) static_cast<T*>(a.out)[static_cast<size_t>(p) * a.ldo + c] = v;
            }
        }
    }
}

template <int DT, int WDT>
__global__ void __launch_bounds__(kThreads) combine_kernel(ExpertArgs a) {
    pdl_wait();
    for (size_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        for (size_t c = threadIdx.x; c < a.cols; c += kThreads) {
            float acc = 0.0f;
            bool first = true;
            for (int j = 0; j < a.topk; ++j) {
                const int p = a.position[t * a.topk + j];
                if (!kept(a, p)) continue;
                const float v = load_elem<DT>(a.rows_in, static_cast<size_t>(p) * a.ldi + c);
                if (a.weights != nullptr) acc = __fmaf_rn(load_elem<WDT>(a.weights, t * a.topk + j), v, acc);
                else acc = first ? v : __fadd_rn(acc, v);
                first = false;
            }
            store_elem<DT>(a.out, t * a.ldo + c, acc);
        }
    }
}

template <int DT, int WDT>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(ExpertArgs a) {
    __shared__ float red[kThreads / 32];
    pdl_wait();
    const size_t n = a.tokens + (a.counts != nullptr ? a.experts : 0);
    for (size_t t = blockIdx.x; t < n; t += gridDim.x) {
        if (t >= a.tokens) {
            if (Elem<DT>::kSize == 4) clear_padding<uint32_t>(a, t - a.tokens);
            else clear_padding<uint16_t>(a, t - a.tokens);
            continue;
        }
        for (int j = 0; j < a.topk; ++j) {
            const size_t slot = t * a.topk + j;
            const int p = a.position[slot];
            float dot = 0.0f;
            if (kept(a, p)) {
                const float w = load_elem<WDT>(a.weights, slot);
                for (size_t c = threadIdx.x; c < a.cols; c += kThreads) {
                    const float d = load_elem<DT>(a.tok, t * a.ldt + c);
                    if (a.dweights != nullptr)
                        dot = __fmaf_rn(d, load_elem<DT>(a.rows_in, static_cast<size_t>(p) * a.ldi + c), dot);
                    store_elem<DT>(a.out, static_cast<size_t>(p) * a.ldo + c, __fmul_rn(w, d));
                }
            }
            if (a.dweights == nullptr) continue;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) dot = __fadd_rn(dot, __shfl_xor_sync(0xFFFFFFFFu, dot, d));
            __syncthreads();
            if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = dot;
            __syncthreads();
            if (threadIdx.x == 0) {
                float s = 0.0f;
                for (int w = 0; w < kThreads / 32; ++w) s = __fadd_rn(s, red[w]);
                store_elem<WDT>(a.dweights, slot, s);
            }
        }
    }
}

unsigned blocks_for(size_t items) { return static_cast<unsigned>(items < 1 ? 1 : (items > (1u << 30) ? 1u << 30 : items)); }

}  // namespace

cudaError_t launch_expert_sort(int id_bytes, const SortArgs& a, cudaStream_t s) {
    const size_t smem = (static_cast<size_t>(kSortWarps) * a.experts + a.experts + 1) * sizeof(int);
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    return launch_kernel_smem(sort_kernel, dim3(1), dim3(kSortThreads), smem, s, a, id_bytes);
}

cudaError_t launch_expert_dispatch(size_t esize, const ExpertArgs& a, cudaStream_t s) {
    const dim3 grid(blocks_for(a.tokens + (a.counts != nullptr ? a.experts : 0)));
    if (esize == 1) return launch_kernel(dispatch_kernel<uint8_t>, grid, dim3(kThreads), s, a);
    if (esize == 2) return launch_kernel(dispatch_kernel<uint16_t>, grid, dim3(kThreads), s, a);
    return launch_kernel(dispatch_kernel<uint32_t>, grid, dim3(kThreads), s, a);
}

cudaError_t launch_expert_combine(sar_dtype dt, sar_dtype wdt, const ExpertArgs& a, cudaStream_t s) {
    const dim3 grid(blocks_for(a.tokens)), block(kThreads);
    switch (dt) {
    case SAR_BF16:
        return wdt == SAR_FP32 ? launch_kernel(combine_kernel<SAR_BF16, SAR_FP32>, grid, block, s, a)
                               : launch_kernel(combine_kernel<SAR_BF16, SAR_BF16>, grid, block, s, a);
    case SAR_FP16:
        return wdt == SAR_FP32 ? launch_kernel(combine_kernel<SAR_FP16, SAR_FP32>, grid, block, s, a)
                               : launch_kernel(combine_kernel<SAR_FP16, SAR_FP16>, grid, block, s, a);
    case SAR_FP32: return launch_kernel(combine_kernel<SAR_FP32, SAR_FP32>, grid, block, s, a);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_expert_combine_backward(sar_dtype dt, sar_dtype wdt, const ExpertArgs& a, cudaStream_t s) {
    const dim3 grid(blocks_for(a.tokens + (a.counts != nullptr ? a.experts : 0))), block(kThreads);
    switch (dt) {
    case SAR_BF16:
        return wdt == SAR_FP32 ? launch_kernel(combine_backward_kernel<SAR_BF16, SAR_FP32>, grid, block, s, a)
                               : launch_kernel(combine_backward_kernel<SAR_BF16, SAR_BF16>, grid, block, s, a);
    case SAR_FP16:
        return wdt == SAR_FP32 ? launch_kernel(combine_backward_kernel<SAR_FP16, SAR_FP32>, grid, block, s, a)
                               : launch_kernel(combine_backward_kernel<SAR_FP16, SAR_FP16>, grid, block, s, a);
    case SAR_FP32: return launch_kernel(combine_backward_kernel<SAR_FP32, SAR_FP32>, grid, block, s, a);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace sar
