// layer_norm.cuh -- the layer norm kernels that keep a row in registers.
//
// A row belongs to a group of TPR threads.  Each thread holds NV vectors of it,
// of VE elements (16 bytes) each, so that the row is read once whatever the
// passes over it.  Two layouts of a row over the group:
//   kVec     vector i of thread t is elements (i * TPR + t) * VE ... + VE - 1,
//            moved as one 16-byte access; rows that all start on 16-byte
//            boundaries with cols a multiple of VE;
//   !kVec    element e of vector i of thread t is (i * VE + e) * TPR + t, moved
//            on its own; a warp's accesses are still contiguous.  Every other
//            row.
#pragma once

#include "sar_device.cuh"
#include "sar_internal.h"

namespace sar {
namespace norm {

// A thread's part of a row: NV vectors as raw bits (16-bit elements in pairs).
template <int DT, int NV> struct Raw { uint4 v[NV]; };

template <int DT, int TPR, int NV, bool kVec>
__device__ __forceinline__ void load_row(Raw<DT, NV>& r, const void* base, size_t first, unsigned t, unsigned cols) {
    constexpr int VE = Elem<DT>::kVE;
    if (kVec) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + first * Elem<DT>::kSize);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const unsigned k = i * TPR + t;
            r.v[i] = k * VE < cols ? ld_stream(p + k) : make_uint4(0, 0, 0, 0);
        }
    } else if (Elem<DT>::kSize == 4) {
        const uint32_t* p = static_cast<const uint32_t*>(base) + first;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const unsigned c = (i * 4 + e) * TPR + t;
                w[e] = c < cols ? p[c] : 0u;
            }
            r.v[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(base) + first;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const unsigned c = (i * 8 + e) * TPR + t;
                h[e] = c < cols ? p[c] : 0u;
            }
            r.v[i] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
        }
    }
}

template <int DT> __device__ __forceinline__ void widen(const uint4& v, float* x) {
    constexpr int W = PerWord<DT>::kN;
    widen_word<DT>(v.x, x);
    widen_word<DT>(v.y, x + W);
    widen_word<DT>(v.z, x + 2 * W);
    widen_word<DT>(v.w, x + 3 * W);
}

// Stores vector i of a row.
template <int DT, int TPR, bool kVec>
__device__ __forceinline__ void store_vec(void* base, size_t first, int i, unsigned t, unsigned cols, const float* x) {
    constexpr int VE = Elem<DT>::kVE, W = PerWord<DT>::kN;
    if (kVec) {
        const unsigned k = i * TPR + t;
        if (k * VE < cols)
            st_stream(reinterpret_cast<uint4*>(static_cast<char*>(base) + first * Elem<DT>::kSize) + k,
                      make_uint4(narrow_word<DT>(x), narrow_word<DT>(x + W), narrow_word<DT>(x + 2 * W),
                                 narrow_word<DT>(x + 3 * W)));
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const unsigned c = (i * VE + e) * TPR + t;
            if (c < cols) store_elem<DT>(base, first + c, x[e]);
        }
    }
}

// Vector i of a parameter (type fp32 or DT; the kVec layout needs it on a
// 16-byte boundary), or `none` where there is no parameter.
template <int DT, int TPR, bool kVec>
__device__ __forceinline__ void load_param(const void* p, bool w32, int i, unsigned t, unsigned cols, float none, float* x) {
    constexpr int VE = Elem<DT>::kVE;
    if (p == nullptr) {
#pragma unroll
        for (int e = 0; e < VE; ++e) x[e] = none;
    } else if (kVec) {
        const unsigned k = i * TPR + t;
        if (k * VE < cols) {
            if (w32) {
                const float4* f = static_cast<const float4*>(p) + k * (VE / 4);
#pragma unroll
                for (int q = 0; q < VE / 4; ++q) {
                    const float4 v = f[q];
                    x[4 * q] = v.x, x[4 * q + 1] = v.y, x[4 * q + 2] = v.z, x[4 * q + 3] = v.w;
                }
            } else {
                widen<DT>(static_cast<const uint4*>(p)[k], x);
            }
        } else {
#pragma unroll
            for (int e = 0; e < VE; ++e) x[e] = none;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const unsigned c = (i * VE + e) * TPR + t;
            x[e] = c >= cols ? none : (w32 ? static_cast<const float*>(p)[c] : load_elem<DT>(p, c));
        }
    }
}

// Whether element e of vector i of thread t is in the row.
template <int DT, int TPR, bool kVec> __device__ __forceinline__ bool in_row(int i, int e, unsigned t, unsigned cols) {
    constexpr int VE = Elem<DT>::kVE;
    return kVec ? (i * TPR + t) * VE < cols : (i * VE + e) * TPR + t < cols;
}

// Sum over the lanes of a group (or over the warp, for groups of warps).
template <int TPR> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int d = (TPR < 32 ? TPR : 32) / 2; d > 0; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

// A barrier among the TPR threads of group g of the block.
template <int TPR, int BT> __device__ __forceinline__ void group_sync(int g) {
    if (TPR == BT) __syncthreads();
    else if (TPR > 32) asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(TPR) : "memory");
}

// ---------------------------------------------------------------------------
// Forward.  Statistics in one exchange between the warps of a group: each warp
// takes its own mean m_w and the deviations' squares q_w around it, and
//   mean = sum s_w / n,   sum (x - mean)^2 = sum (q_w + n_w (m_w - mean)^2),
// which keeps the digits that sum x^2 - n mean^2 would lose.
// ---------------------------------------------------------------------------
template <int DT, int TPR, int NV, bool kVec>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) forward_kernel(NormArgs a, bool w32) {
    constexpr int VE = Elem<DT>::kVE, BT = TPR < 128 ? 128 : TPR, RPB = BT / TPR, WPG = TPR > 32 ? TPR / 32 : 1;
    __shared__ float4 red[TPR > 32 ? WPG : 1];
    pdl_wait();
    const unsigned t = threadIdx.x % TPR, cols = static_cast<unsigned>(a.cols);
    const size_t groups = static_cast<size_t>(gridDim.x) * RPB;
    // All threads of a block make the same number of rounds.
    for (size_t r0 = static_cast<size_t>(blockIdx.x) * RPB; r0 < a.rows; r0 += groups) {
        const size_t r = r0 + threadIdx.x / TPR;
        const bool live = RPB == 1 || r < a.rows;
        Raw<DT, NV> x;
        load_row<DT, TPR, NV, kVec>(x, a.x, live ? r * a.ldx : 0, t, live ? cols : 0u);
        float s = 0.0f, have = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[VE];
            widen<DT>(x.v[i], f);
#pragma unroll
            for (int e = 0; e < VE; ++e) s = __fadd_rn(s, f[e]);
        }
        // Elements of this warp (or group of lanes): whole warps but the last.
        if (TPR > 32) {
            unsigned n = 0;
#pragma unroll
            for (int i = 0; i < NV * (kVec ? 1 : VE); ++i) {
                const unsigned from = (i * TPR + (t & ~31u)) * (kVec ? VE : 1);
                const unsigned left = from < cols ? cols - from : 0u;
                n += left < 32u * (kVec ? VE : 1) ? left : 32u * (kVec ? VE : 1);
            }
            have = static_cast<float>(n);
        } else {
            have = static_cast<float>(cols);
        }
        s = lanes_sum<TPR>(s);
        float mean = have > 0.0f ? s / have : 0.0f;
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[VE];
            widen<DT>(x.v[i], f);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float d = __fsub_rn(f[e], mean);
                if (in_row<DT, TPR, kVec>(i, e, t, cols)) q = __fmaf_rn(d, d, q);
            }
        }
        q = lanes_sum<TPR>(q);
        const float n = static_cast<float>(cols);
        if (TPR > 32) {
            if ((t & 31) == 0) red[t / 32] = make_float4(s, q, mean, have);
            group_sync<TPR, BT>(0);
            if (WPG <= 8) {
                s = 0.0f;
#pragma unroll
                for (int w = 0; w < WPG; ++w) s = __fadd_rn(s, red[w].x);
                mean = s / n;
                q = 0.0f;
#pragma unroll
                for (int w = 0; w < WPG; ++w) {
                    const float d = __fsub_rn(red[w].z, mean);
                    q = __fadd_rn(q, __fmaf_rn(__fmul_rn(red[w].w, d), d, red[w].y));
                }
            } else {
                const float4 p = red[(t & 31) % WPG];
                s = p.x;
#pragma unroll
                for (int d = WPG / 2; d > 0; d >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, d));
                mean = s / n;
                const float d0 = __fsub_rn(p.z, mean);
                q = __fmaf_rn(__fmul_rn(p.w, d0), d0, p.y);
#pragma unroll
                for (int d = WPG / 2; d > 0; d >>= 1) q = __fadd_rn(q, __shfl_xor_sync(0xFFFFFFFFu, q, d));
            }
        }
        const float rstd = 1.0f / sqrtf(q / n + a.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[VE], w[VE], b[VE];
            load_param<DT, TPR, kVec>(a.weight, w32, i, t, cols, 1.0f, w);
            load_param<DT, TPR, kVec>(a.bias, w32, i, t, cols, 0.0f, b);
            widen<DT>(x.v[i], f);
#pragma unroll
            for (int e = 0; e < VE; ++e) f[e] = __fmaf_rn(__fmul_rn(__fsub_rn(f[e], mean), rstd), w[e], b[e]);
            store_vec<DT, TPR, kVec>(a.y, live ? r * a.ldy : 0, i, t, live ? cols : 0u, f);
        }
        if (live && t == 0) {
            if (a.mean != nullptr) a.mean[r] = mean;
            if (a.rstd != nullptr) a.rstd[r] = rstd;
        }
        if (TPR > 32) group_sync<TPR, BT>(0);       // red is free again
    }
}

// ---------------------------------------------------------------------------
// Backward.  Blocks stay for many rows; every thread adds dy * h and dy of its
// columns up in registers, row after row, while the next row's loads are in
// flight.  At the end the groups of a block are added in order in shared
// memory, and each block writes one row of sums, which params_kernel adds.
// ---------------------------------------------------------------------------
constexpr int kSMs = 152;

template <int TPR> struct BackwardShape {
    static constexpr int kThreads = TPR > 512 ? TPR : 512;
    static constexpr int kGroups = kThreads / TPR;
};

template <int DT, int TPR, int NV, bool kVec>
__global__ void __launch_bounds__(BackwardShape<TPR>::kThreads, NV == 1 && TPR <= 512 ? 2 : 1)
backward_kernel(NormGradArgs a, bool w32) {
    constexpr int VE = Elem<DT>::kVE, BT = BackwardShape<TPR>::kThreads, G = BT / TPR, WPG = TPR > 32 ? TPR / 32 : 1;
    __shared__ float2 red[2][G][WPG];
    extern __shared__ float sums[];                   // [G][2][NV * TPR * VE], groups of at least a warp
    pdl_wait();
    const unsigned t = threadIdx.x % TPR, cols = static_cast<unsigned>(a.cols);
    const int g = threadIdx.x / TPR;
    const size_t step = static_cast<size_t>(gridDim.x) * G;
    const float n = static_cast<float>(cols);
    float dw[NV * VE], db[NV * VE];
#pragma unroll
    for (int e = 0; e < NV * VE; ++e) dw[e] = db[e] = 0.0f;
    Raw<DT, NV> x, dy;
    float mean = 0.0f, rstd = 0.0f;
    // Groups smaller than a warp keep its lanes together: the warp makes the
    // rounds of its first group, lanes without a row on zeros.
    const size_t first = static_cast<size_t>(blockIdx.x) * G;
    size_t r = first + g, lead = first + (TPR < 32 ? (threadIdx.x & ~31u) / TPR : g);
    auto fetch = [&] {
        const bool live = r < a.rows;
        load_row<DT, TPR, NV, kVec>(x, a.x, live ? r * a.ldx : 0, t, live ? cols : 0u);
        load_row<DT, TPR, NV, kVec>(dy, a.dy, live ? r * a.lddy : 0, t, live ? cols : 0u);
        mean = live ? a.mean[r] : 0.0f;
        rstd = live ? a.rstd[r] : 0.0f;
    };
    fetch();
    for (int buf = 0; lead < a.rows; lead += step, buf ^= 1) {
        const size_t row = r;
        const Raw<DT, NV> cx = x, cdy = dy;
        const float m = mean, rs = rstd;
        r += step;
        if (NV == 1) fetch();
        float s = 0.0f, q = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float fx[VE], fd[VE], w[VE];
            widen<DT>(cx.v[i], fx);
            widen<DT>(cdy.v[i], fd);
            load_param<DT, TPR, kVec>(a.weight, w32, i, t, cols, 1.0f, w);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float h = __fmul_rn(__fsub_rn(fx[e], m), rs), gr = __fmul_rn(fd[e], w[e]);
                s = __fadd_rn(s, gr);
                q = __fmaf_rn(gr, h, q);
                dw[i * VE + e] = __fmaf_rn(fd[e], h, dw[i * VE + e]);
                db[i * VE + e] = __fadd_rn(db[i * VE + e], fd[e]);
            }
        }
        s = lanes_sum<TPR>(s);
        q = lanes_sum<TPR>(q);
        if (TPR > 32) {
            if ((t & 31) == 0) red[buf][g][t / 32] = make_float2(s, q);
            group_sync<TPR, BT>(g);
            const float2 p = red[buf][g][(t & 31) % WPG];
            s = p.x, q = p.y;
#pragma unroll
            for (int d = WPG / 2; d > 0; d >>= 1) {
                s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, d));
                q = __fadd_rn(q, __shfl_xor_sync(0xFFFFFFFFu, q, d));
            }
        }
        const float mg = s / n, mgh = q / n;
        const bool live = row < a.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float fx[VE], fd[VE], w[VE];
            widen<DT>(cx.v[i], fx);
            widen<DT>(cdy.v[i], fd);
            load_param<DT, TPR, kVec>(a.weight, w32, i, t, cols, 1.0f, w);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float h = __fmul_rn(__fsub_rn(fx[e], m), rs), gr = __fmul_rn(fd[e], w[e]);
                fx[e] = __fmul_rn(rs, __fmaf_rn(-h, mgh, __fsub_rn(gr, mg)));
            }
            store_vec<DT, TPR, kVec>(a.dx, live ? row * a.lddx : 0, i, t, live ? cols : 0u, fx);
        }
        if (NV != 1) fetch();
    }
    if (a.dweight == nullptr && a.dbias == nullptr) return;
    float* out = a.partial + static_cast<size_t>(blockIdx.x) * 2 * cols;
    if (G == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const unsigned c = kVec ? (i * TPR + t) * VE + e : (i * VE + e) * TPR + t;
                if (c < cols) {
                    out[c] = dw[i * VE + e];
                    out[cols + c] = db[i * VE + e];
                }
            }
        return;
    }
    constexpr int C = NV * TPR * VE, S = TPR < 32 ? BT / 32 : G;
    if (TPR < 32) {
#pragma unroll
        for (int e = 0; e < NV * VE; ++e)
#pragma unroll
            for (int d = TPR; d < 32; d <<= 1) {
                dw[e] = __fadd_rn(dw[e], __shfl_xor_sync(0xFFFFFFFFu, dw[e], d));
                db[e] = __fadd_rn(db[e], __shfl_xor_sync(0xFFFFFFFFu, db[e], d));
            }
    }
    const int slot = TPR < 32 ? threadIdx.x / 32 : g;
    if (TPR >= 32 || (threadIdx.x & 31) < TPR) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const unsigned c = kVec ? (i * TPR + t) * VE + e : (i * VE + e) * TPR + t;
                sums[(slot * 2) * C + c] = dw[i * VE + e];
                sums[(slot * 2 + 1) * C + c] = db[i * VE + e];
            }
    }
    __syncthreads();
    for (unsigned c = threadIdx.x; c < 2 * cols; c += BT) {
        const unsigned half = c >= cols, k = half * C + (c - half * cols);
        float v = sums[k];
        for (int p = 1; p < S; ++p) v = __fadd_rn(v, sums[p * 2 * C + k]);
        out[c] = v;
    }
}

// Threads per row of the backward kernel for a row of `vecs` vectors, and its
// vectors per thread (0: the row does not fit the registers).
inline int backward_tpr(size_t vecs) {
    int tpr = 8;
    while (tpr < 1024 && static_cast<size_t>(tpr) < vecs) tpr *= 2;
    return tpr;
}

template <int DT> cudaError_t forward(const NormArgs& a, bool w32, bool vec, cudaStream_t s);
template <int DT> cudaError_t backward(const NormGradArgs& a, bool w32, bool vec, unsigned blocks, cudaStream_t s);

template <int DT, int TPR, int NV>
cudaError_t forward_launch(const NormArgs& a, bool w32, bool vec, cudaStream_t s) {
    constexpr int BT = TPR < 128 ? 128 : TPR, RPB = BT / TPR;
    const size_t blocks = (a.rows + RPB - 1) / RPB;
    const dim3 grid(static_cast<unsigned>(blocks < 0x7FFFFFFF ? blocks : 0x7FFFFFFF));
    return vec ? launch_kernel(forward_kernel<DT, TPR, NV, true>, grid, dim3(BT), s, a, w32)
               : launch_kernel(forward_kernel<DT, TPR, NV, false>, grid, dim3(BT), s, a, w32);
}

template <int DT, int TPR, int NV>
cudaError_t backward_launch(const NormGradArgs& a, bool w32, bool vec, unsigned blocks, cudaStream_t s) {
    constexpr int BT = BackwardShape<TPR>::kThreads, G = BT / TPR, S = TPR < 32 ? BT / 32 : G;
    const size_t smem = G == 1 ? 0 : static_cast<size_t>(S) * 2 * NV * TPR * Elem<DT>::kVE * sizeof(float);
    return vec ? launch_kernel_smem(backward_kernel<DT, TPR, NV, true>, dim3(blocks), dim3(BT), smem, s, a, w32)
               : launch_kernel_smem(backward_kernel<DT, TPR, NV, false>, dim3(blocks), dim3(BT), smem, s, a, w32);
}

// Definitions for one element type (layer_norm_<type>.cu).
template <int DT> cudaError_t forward_any(const NormArgs& a, bool w32, bool vec, cudaStream_t s) {
    const size_t vecs = (a.cols + Elem<DT>::kVE - 1) / Elem<DT>::kVE;
    if (vecs <= 8) return forward_launch<DT, 8, 1>(a, w32, vec, s);
    if (vecs <= 32) return forward_launch<DT, 32, 1>(a, w32, vec, s);
    if (vecs <= 64) return forward_launch<DT, 32, 2>(a, w32, vec, s);
    if (vecs <= 128) return forward_launch<DT, 32, 4>(a, w32, vec, s);
    if (vecs <= 256) return forward_launch<DT, 128, 2>(a, w32, vec, s);
    if (vecs <= 512) return forward_launch<DT, 128, 4>(a, w32, vec, s);
    if (vecs <= 1024) return forward_launch<DT, 256, 4>(a, w32, vec, s);
    if (vecs <= 2048) return forward_launch<DT, 512, 4>(a, w32, vec, s);
    if (vecs <= 4096) return forward_launch<DT, 1024, 4>(a, w32, vec, s);
    if (vecs <= 8192) return forward_launch<DT, 1024, 8>(a, w32, vec, s);
    return cudaErrorInvalidValue;
}

template <int DT> cudaError_t backward_any(const NormGradArgs& a, bool w32, bool vec, unsigned blocks, cudaStream_t s) {
    switch (backward_tpr((a.cols + Elem<DT>::kVE - 1) / Elem<DT>::kVE)) {
    case 8: return backward_launch<DT, 8, 1>(a, w32, vec, blocks, s);
    case 16: return backward_launch<DT, 16, 1>(a, w32, vec, blocks, s);
    case 32: return backward_launch<DT, 32, 1>(a, w32, vec, blocks, s);
    case 64: return backward_launch<DT, 64, 1>(a, w32, vec, blocks, s);
    case 128: return backward_launch<DT, 128, 1>(a, w32, vec, blocks, s);
    case 256: return backward_launch<DT, 256, 1>(a, w32, vec, blocks, s);
    case 512: return backward_launch<DT, 512, 1>(a, w32, vec, blocks, s);
    default: return backward_launch<DT, 1024, 1>(a, w32, vec, blocks, s);
    }
}

}  // namespace norm
}  // namespace sar
