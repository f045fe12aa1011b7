// expert_layer.cu -- the whole expert layer of a few tokens.
#include "sar_device.cuh"
#include "sar_internal.h"

namespace sar {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
    return x;
}

__device__ __forceinline__ float activate(float z, sar_activation act) {
    if (act == SAR_ACT_SILU) return __fdiv_rn(z, __fadd_rn(1.0f, expf(-z)));
    if (act == SAR_ACT_GELU) return __fmul_rn(__fmul_rn(0.5f, z), erfcf(__fmul_rn(z, -0.70710678f)));
    return z <= 0.0f ? 0.0f : z;
}

template <int DT> __device__ float dot(const void* w, size_t at, const void* x, size_t xat, int n, int lane) {
    float s = 0.0f;
    for (int k = lane; k < n; k += 32) s = __fmaf_rn(load_elem<DT>(w, at + k), load_elem<DT>(x, xat + k), s);
    return warp_sum(s);
}

__device__ __forceinline__ int expert_of(const void* ids, int id_bytes, int slot, int experts) {
    const int64_t e = id_bytes == 8 ? static_cast<const int64_t*>(ids)[slot] : static_cast<const int32_t*>(ids)[slot];
    return e >= 0 && e < experts ? static_cast<int>(e) : -1;
}

template <int DT> __global__ void in_kernel(LayerArgs a, int id_bytes) {
    pdl_wait();
    const int lane = threadIdx.x & 31, i = blockIdx.x * kWarps + (threadIdx.x >> 5), slot = blockIdx.y;
    const int e = expert_of(a.ids, id_bytes, slot, a.experts);
    if (i >= a.hidden || e < 0) return;
    const size_t rows = static_cast<size_t>(a.gated ? 2 : 1) * a.hidden, k = a.cols, xat = (slot / a.topk) * a.ldx;
    const float z = dot<DT>(a.w_in, (e * rows + i) * k, a.x, xat, a.cols, lane);
    float h = activate(z, a.activation);
    if (a.gated) h = __fmul_rn(h, dot<DT>(a.w_in, (e * rows + a.hidden + i) * k, a.x, xat, a.cols, lane));
    if (lane == 0) static_cast<float*>(a.workspace)[static_cast<size_t>(slot) * a.hidden + i] = h;
}

template <int DT, int WDT> __global__ void out_kernel(LayerArgs a, int id_bytes) {
    pdl_wait();
    const int lane = threadIdx.x & 31, c = blockIdx.x * kWarps + (threadIdx.x >> 5), t = blockIdx.y;
    if (c >= a.cols) return;
    float total = 0.0f;
    for (int j = 0; j < a.topk; ++j) {
        const int slot = t * a.topk + j, e = expert_of(a.ids, id_bytes, slot, a.experts);
        if (e < 0) continue;
        float s = 0.0f;
        const float* h = static_cast<const float*>(a.workspace) + static_cast<size_t>(slot) * a.hidden;
        for (int k = lane; k < a.hidden; k += 32)
            s = __fmaf_rn(load_elem<DT>(a.w_out, (static_cast<size_t>(e) * a.cols + c) * a.hidden + k), h[k], s);
        s = warp_sum(s);
        total = __fmaf_rn(a.weights != nullptr ? load_elem<WDT>(a.weights, slot) : 1.0f, s, total);
    }
    if (lane == 0) store_elem<DT>(a.out, t * a.ldo + c, total);
}

template <int DT, int WDT> cudaError_t launch(int id_bytes, const LayerArgs& a, cudaStream_t s) {
    const dim3 block(kWarps * 32);
    if (a.hidden > 0) {
        const cudaError_t e = launch_kernel(in_kernel<DT>, dim3((a.hidden + kWarps - 1) / kWarps, a.tokens * a.topk), block, s,
                                            a, id_bytes);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(out_kernel<DT, WDT>, dim3((a.cols + kWarps - 1) / kWarps, a.tokens), block, s, a, id_bytes);
}

}  // namespace

size_t expert_layer_workspace_bytes(size_t slots, size_t, size_t hidden) { return 16 + slots * hidden * 4; }

cudaError_t launch_expert_layer(sar_dtype dt, sar_dtype wdt, int id_bytes, const LayerArgs& a, cudaStream_t s) {
    switch (dt) {
    case SAR_BF16: return wdt == SAR_FP32 ? launch<SAR_BF16, SAR_FP32>(id_bytes, a, s) : launch<SAR_BF16, SAR_BF16>(id_bytes, a, s);
    case SAR_FP16: return wdt == SAR_FP32 ? launch<SAR_FP16, SAR_FP32>(id_bytes, a, s) : launch<SAR_FP16, SAR_FP16>(id_bytes, a, s);
    default: return launch<SAR_FP32, SAR_FP32>(id_bytes, a, s);
    }
}

}  // namespace sar
