// orthogonalize.cu -- Newton-Schulz iteration of a batch of matrices.
#include <algorithm>

#include "sar_device.cuh"
#include "sar_internal.h"

namespace sar {
namespace {

constexpr int kNormThreads = 256;
constexpr size_t kMaxParts = 256;

size_t norm_parts(size_t rows, size_t cols) { return std::min(kMaxParts, std::max<size_t>(1, rows * cols / 16384)); }

// Sums of squares whatever the values' magnitude: those that would overflow or
// vanish are scaled, each kind in a sum of its own.
struct Squares {
    float big = 0.0f, mid = 0.0f, small = 0.0f;
    __device__ __forceinline__ void add(float x) {
        const float m = fabsf(x);
        if (m > 0x1p45f) {
            const float y = x * 0x1p-90f;
            big = __fmaf_rn(y, y, big);
        } else if (m < 0x1p-40f) {
            const float y = x * 0x1p80f;
            small = __fmaf_rn(y, y, small);
        } else {
            mid = __fmaf_rn(x, x, mid);
        }
    }
};

__device__ __forceinline__ float block_sum(float x, float* shared) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < kNormThreads / 32; ++w) s = __fadd_rn(s, shared[w]);
    return s;
}

// parts x 3 sums for each matrix.
template <int DT> __global__ void __launch_bounds__(kNormThreads) squares_kernel(OrthogonalizeArgs a, float* sums) {
    pdl_wait();
    __shared__ float shared[kNormThreads / 32];
    const size_t z = blockIdx.y, count = a.rows * a.cols, threads = static_cast<size_t>(gridDim.x) * kNormThreads;
    Squares q;
    for (size_t i = static_cast<size_t>(blockIdx.x) * kNormThreads + threadIdx.x; i < count; i += threads)
        q.add(load_elem<DT>(a.g, z * a.gstride + i / a.cols * a.ldg + i % a.cols));
    const float big = block_sum(q.big, shared), mid = block_sum(q.mid, shared), small = block_sum(q.small, shared);
    if (threadIdx.x == 0) {
        float* out = sums + (z * gridDim.x + blockIdx.x) * 3;
        out[0] = big, out[1] = mid, out[2] = small;
    }
}

// 1 / (norm + eps) = f * first * second, both of the latter powers of two: none
// of them leaves binary32's range.
struct Factor {
    float f, first, second;
    __device__ __forceinline__ float of(float x) const { return x * first * f * second; }
};

__device__ Factor factor(const float* sums, int parts, float eps) {
    double total = 0.0;
    for (int i = 0; i < parts; ++i)
        total += static_cast<double>(sums[3 * i]) * 0x1p180 + sums[3 * i + 1] + static_cast<double>(sums[3 * i + 2]) * 0x1p-160;
    const double inv = 1.0 / (sqrt(total) + static_cast<double>(eps));
    if (!(inv > 0.0) || isinf(inv)) return {static_cast<float>(inv), 1.0f, 1.0f};
    int e;
    const double f = frexp(inv, &e);
    return {static_cast<float>(f), ldexpf(1.0f, e / 2), ldexpf(1.0f, e - e / 2)};
}

template <int DT> __global__ void __launch_bounds__(256) begin_kernel(OrthogonalizeArgs a, const float* sums, int parts, float* x) {
    pdl_wait();
    __shared__ Factor f;
    const size_t z = blockIdx.y, count = a.rows * a.cols;
    if (threadIdx.x == 0) f = factor(sums + z * parts * 3, parts, a.eps);
    __syncthreads();
    const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= count) return;
    const size_t r = i / a.cols, c = i % a.cols;
    const float v = f.of(load_elem<DT>(a.g, z * a.gstride + r * a.ldg + c));
    x[z * count + (a.rows > a.cols ? c * a.rows + r : i)] = v;
}

template <int DT> __global__ void __launch_bounds__(256) end_kernel(OrthogonalizeArgs a, const float* x) {
    pdl_wait();
    const size_t z = blockIdx.y, count = a.rows * a.cols, i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= count) return;
    const size_t r = i / a.cols, c = i % a.cols;
    store_elem<DT>(a.out, z * a.ostride + r * a.ldo + c, a.scale * x[z * count + (a.rows > a.cols ? c * a.rows + r : i)]);
}

// C = alpha * (P Q or P Q^T) + beta * D, all dense; P is m x k.
template <bool TRANSPOSED>
__global__ void __launch_bounds__(256) product_kernel(const float* P, const float* Q, const float* D, float* C, int m, int n, int k,
                                                      float alpha, float beta, size_t sp, size_t sq, size_t sc) {
    pdl_wait();
    __shared__ float p[16][65], q[16][65];
    P += blockIdx.z * sp, Q += blockIdx.z * sq, C += blockIdx.z * sc;
    if (D != nullptr) D += blockIdx.z * sc;
    const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64, t = threadIdx.x, tr = t / 16, tc = t % 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < k; k0 += 16) {
        for (int i = t; i < 1024; i += 256) {
            const int row = i / 16, kk = i % 16;
            p[kk][row] = r0 + row < m && k0 + kk < k ? P[static_cast<size_t>(r0 + row) * k + k0 + kk] : 0.0f;
            if (TRANSPOSED) {
                q[kk][row] = c0 + row < n && k0 + kk < k ? Q[static_cast<size_t>(c0 + row) * k + k0 + kk] : 0.0f;
            } else {
                const int col = i % 64, kq = i / 64;
                q[kq][col] = c0 + col < n && k0 + kq < k ? Q[static_cast<size_t>(k0 + kq) * n + c0 + col] : 0.0f;
            }
        }
        __syncthreads();
        for (int kk = 0; kk < 16; ++kk)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = __fmaf_rn(p[kk][tr * 4 + i], q[kk][tc * 4 + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int r = r0 + tr * 4 + i, c = c0 + tc * 4 + j;
            if (r < m && c < n) {
                const size_t at = static_cast<size_t>(r) * n + c;
                C[at] = __fadd_rn(__fmul_rn(alpha, acc[i][j]), D != nullptr ? __fmul_rn(beta, D[at]) : 0.0f);
            }
        }
}

template <int DT> cudaError_t launch(const OrthogonalizeArgs& a, cudaStream_t s) {
    const size_t small = std::min(a.rows, a.cols), large = std::max(a.rows, a.cols), count = small * large, sq = small * small;
    const unsigned parts = static_cast<unsigned>(norm_parts(a.rows, a.cols)), batch = static_cast<unsigned>(a.batch);
    float* sums = static_cast<float*>(a.workspace);
    float *x = sums + a.batch * kMaxParts * 4, *y = x + a.batch * count, *gram = y + a.batch * count, *poly = gram + a.batch * sq;
    const dim3 all(static_cast<unsigned>((count + 255) / 256), batch);
    cudaError_t e = launch_kernel(squares_kernel<DT>, dim3(parts, batch), dim3(kNormThreads), s, a, sums);
    if (e == cudaSuccess) e = launch_kernel(begin_kernel<DT>, all, dim3(256), s, a, static_cast<const float*>(sums),
                                            static_cast<int>(parts), x);
    const int m = static_cast<int>(small), n = static_cast<int>(large);
    const dim3 gm((m + 63) / 64, (m + 63) / 64, batch), gx((n + 63) / 64, (m + 63) / 64, batch);
    for (int k = 0; k < a.steps && e == cudaSuccess; ++k) {
        e = launch_kernel(product_kernel<true>, gm, dim3(256), s, x, x, static_cast<const float*>(nullptr), gram, m, m, n, 1.0f,
                          0.0f, count, count, sq);
        if (e == cudaSuccess) e = launch_kernel(product_kernel<true>, gm, dim3(256), s, gram, gram, gram, poly, m, m, m, a.c, a.b, sq, sq, sq);
        if (e == cudaSuccess) e = launch_kernel(product_kernel<false>, gx, dim3(256), s, poly, x, x, y, m, n, m, 1.0f, a.a, sq, count, count);
        std::swap(x, y);
    }
    if (e == cudaSuccess) e = launch_kernel(end_kernel<DT>, all, dim3(256), s, a, static_cast<const float*>(x));
    return e;
}

}  // namespace

size_t orthogonalize_workspace_bytes(size_t batch, size_t rows, size_t cols) {
    const size_t small = std::min(rows, cols);
    return 16 + batch * 4 * (kMaxParts * 4 + 2 * rows * cols + 2 * small * small);
}

cudaError_t launch_orthogonalize(sar_dtype dt, const OrthogonalizeArgs& a, cudaStream_t s) {
    switch (dt) {
    case SAR_BF16: return launch<SAR_BF16>(a, s);
    case SAR_FP16: return launch<SAR_FP16>(a, s);
    default: return launch<SAR_FP32>(a, s);
    }
}

}  // namespace sar
