// layer_norm.cu -- layer norm and its gradient.
//
// Forward, per row of C elements:  mean = sum x / C,  var = sum (x - mean)^2 / C,
// rstd = 1 / sqrt(var + eps),  y = (x - mean) rstd w + b.  Backward, with
// h = (x - mean) rstd and g = dy w:  dx = rstd (g - mean(g) - h mean(g h)),
// dw = sum over rows of dy h,  db = sum over rows of dy.
//
// First form: one block per row, element by element; the parameters' gradients
// in a kernel of their own, a thread per column over a share of the rows, and
// a second one that adds the shares in order.
#include "sar_device.cuh"
#include "sar_internal.h"

namespace sar {
namespace {

constexpr size_t kShares = 64;

template <int WDT> __device__ __forceinline__ float param(const void* p, size_t i, float none) {
    return p != nullptr ? load_elem<WDT>(p, i) : none;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

// The block's sum in every thread; `red` holds one value per warp.
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (unsigned w = 0; w < blockDim.x >> 5; ++w) s = __fadd_rn(s, red[w]);
    return s;
}

template <int DT, int WDT>
__global__ void __launch_bounds__(kThreads) norm_rows_kernel(NormArgs a) {
    __shared__ float red[kThreads / 32];
    pdl_wait();
    const float n = static_cast<float>(a.cols);
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const size_t bx = r * a.ldx, by = r * a.ldy;
        float s = 0.0f;
        for (size_t c = threadIdx.x; c < a.cols; c += kThreads) s = __fadd_rn(s, load_elem<DT>(a.x, bx + c));
        const float mean = block_sum(s, red) / n;
        float q = 0.0f;
        for (size_t c = threadIdx.x; c < a.cols; c += kThreads) {
            const float d = __fsub_rn(load_elem<DT>(a.x, bx + c), mean);
            q = __fmaf_rn(d, d, q);
        }
        const float rstd = 1.0f / sqrtf(block_sum(q, red) / n + a.eps);
        for (size_t c = threadIdx.x; c < a.cols; c += kThreads) {
            const float h = __fmul_rn(__fsub_rn(load_elem<DT>(a.x, bx + c), mean), rstd);
            store_elem<DT>(a.y, by + c, __fmaf_rn(h, param<WDT>(a.weight, c, 1.0f), param<WDT>(a.bias, c, 0.0f)));
        }
        if (threadIdx.x == 0) {
            if (a.mean != nullptr) a.mean[r] = mean;
            if (a.rstd != nullptr) a.rstd[r] = rstd;
        }
    }
}

template <int DT, int WDT>
__global__ void __launch_bounds__(kThreads) norm_dx_kernel(NormGradArgs a) {
    __shared__ float red[kThreads / 32];
    pdl_wait();
    const float n = static_cast<float>(a.cols);
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const size_t bx = r * a.ldx, bd = r * a.lddy, bo = r * a.lddx;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s = 0.0f, q = 0.0f;
        for (size_t c = threadIdx.x; c < a.cols; c += kThreads) {
            const float h = __fmul_rn(__fsub_rn(load_elem<DT>(a.x, bx + c), mean), rstd);
            const float g = __fmul_rn(load_elem<DT>(a.dy, bd + c), param<WDT>(a.weight, c, 1.0f));
            s = __fadd_rn(s, g);
            q = __fmaf_rn(g, h, q);
        }
        const float mg = block_sum(s, red) / n, mgh = block_sum(q, red) / n;
        for (size_t c = threadIdx.x; c < a.cols; c += kThreads) {
            const float h = __fmul_rn(__fsub_rn(load_elem<DT>(a.x, bx + c), mean), rstd);
            const float g = __fmul_rn(load_elem<DT>(a.dy, bd + c), param<WDT>(a.weight, c, 1.0f));
            store_elem<DT>(a.dx, bo + c, __fmul_rn(rstd, __fmaf_rn(-h, mgh, __fsub_rn(g, mg))));
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) norm_shares_kernel(NormGradArgs a) {
    pdl_wait();
    const size_t shares = gridDim.y, per = (a.rows + shares - 1) / shares;
    const size_t r0 = per * blockIdx.y, r1 = r0 + per < a.rows ? r0 + per : a.rows;
    for (size_t c = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x; c < a.cols;
         c += static_cast<size_t>(gridDim.x) * kThreads) {
        float w = 0.0f, b = 0.0f;
        for (size_t r = r0; r < r1; ++r) {
            const float d = load_elem<DT>(a.dy, r * a.lddy + c);
            const float h = __fmul_rn(__fsub_rn(load_elem<DT>(a.x, r * a.ldx + c), a.mean[r]), a.rstd[r]);
            w = __fmaf_rn(d, h, w);
            b = __fadd_rn(b, d);
        }
        a.partial[blockIdx.y * 2 * a.cols + c] = w;
        a.partial[(blockIdx.y * 2 + 1) * a.cols + c] = b;
    }
}

template <int WDT>
__global__ void __launch_bounds__(kThreads) norm_params_kernel(NormGradArgs a, size_t shares) {
    pdl_wait();
    for (size_t c = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x; c < a.cols;
         c += static_cast<size_t>(gridDim.x) * kThreads) {
        float w = 0.0f, b = 0.0f;
        for (size_t k = 0; k < shares; ++k) {
            w = __fadd_rn(w, a.partial[k * 2 * a.cols + c]);
            b = __fadd_rn(b, a.partial[(k * 2 + 1) * a.cols + c]);
        }
        if (a.dweight != nullptr) store_elem<WDT>(a.dweight, c, w);
        if (a.dbias != nullptr) store_elem<WDT>(a.dbias, c, b);
    }
}

unsigned blocks_for(size_t items, size_t per, size_t cap) {
    const size_t g = (items + per - 1) / per;
    return static_cast<unsigned>(g < 1 ? 1 : (g > cap ? cap : g));
}

template <int DT, int WDT> cudaError_t norm(const NormArgs& a, cudaStream_t s) {
    return launch_kernel(norm_rows_kernel<DT, WDT>, dim3(blocks_for(a.rows, 1, 1u << 30)), dim3(kThreads), s, a);
}

template <int DT, int WDT> cudaError_t norm_backward(const NormGradArgs& a, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (a.dweight != nullptr || a.dbias != nullptr) {
        const size_t shares = layer_norm_partials(a.rows, a.cols);
        const unsigned gx = blocks_for(a.cols, kThreads, 1024);
        e = launch_kernel(norm_shares_kernel<DT>, dim3(gx, static_cast<unsigned>(shares)), dim3(kThreads), s, a);
        if (e != cudaSuccess) return e;
        e = launch_kernel(norm_params_kernel<WDT>, dim3(gx), dim3(kThreads), s, a, shares);
        if (e != cudaSuccess || a.rows == 0) return e;
    }
    return launch_kernel(norm_dx_kernel<DT, WDT>, dim3(blocks_for(a.rows, 1, 1u << 30)), dim3(kThreads), s, a);
}

}  // namespace

size_t layer_norm_partials(size_t rows, size_t) { return rows < 1 ? 1 : (rows < kShares ? rows : kShares); }

cudaError_t launch_layer_norm(sar_dtype dt, sar_dtype wdt, const NormArgs& a, cudaStream_t s) {
    switch (dt) {
    case SAR_BF16: return wdt == SAR_FP32 ? norm<SAR_BF16, SAR_FP32>(a, s) : norm<SAR_BF16, SAR_BF16>(a, s);
    case SAR_FP16: return wdt == SAR_FP32 ? norm<SAR_FP16, SAR_FP32>(a, s) : norm<SAR_FP16, SAR_FP16>(a, s);
    case SAR_FP32: return norm<SAR_FP32, SAR_FP32>(a, s);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_layer_norm_backward(sar_dtype dt, sar_dtype wdt, const NormGradArgs& a, cudaStream_t s) {
    switch (dt) {
    case SAR_BF16:
        return wdt == SAR_FP32 ? norm_backward<SAR_BF16, SAR_FP32>(a, s) : norm_backward<SAR_BF16, SAR_BF16>(a, s);
    case SAR_FP16:
        return wdt == SAR_FP32 ? norm_backward<SAR_FP16, SAR_FP32>(a, s) : norm_backward<SAR_FP16, SAR_FP16>(a, s);
    case SAR_FP32: return norm_backward<SAR_FP32, SAR_FP32>(a, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace sar
