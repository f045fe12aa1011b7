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
// These kernels take the calls of few rows, where a launch and one pass of
// latency are what counts (8 x 4096 bf16 forward 2.0 us, 100 x 1024 backward 1.9
// without the parameters' gradients and 4.6 with), rows of up to 16 vectors, and
// matrices whose rows do not start alike (a slice of 1021 of 1024 columns with a
// dense output, 16384 rows bf16: forward 58 us, where rows that do take 24);
// layer_norm_ring.cuh has the ones for many rows.  Rows of over 4096 vectors, eight
// a thread, do not fit 64 registers and spill 192 to 276 bytes a thread.
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
            r.v[i] = k * VE < cols ? ld_stream_ordered(p + k) : make_uint4(0, 0, 0, 0);
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

// Arithmetic on pairs of elements: one instruction for two (add, mul and fma on
// .f32x2, each half rounded as the scalar one).  The kernels below issue close
// to what the SMs can while HBM streams, so the count matters.
__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }

// A vector's elements in pairs, in binary32.
template <int DT> __device__ __forceinline__ void widen(const uint4& v, float2* x) {
    constexpr int W = PerWord<DT>::kN;
    float f[4 * W];
    widen_word<DT>(v.x, f);
    widen_word<DT>(v.y, f + W);
    widen_word<DT>(v.z, f + 2 * W);
    widen_word<DT>(v.w, f + 3 * W);
#pragma unroll
    for (int p = 0; p < 2 * W; ++p) x[p] = make_float2(f[2 * p], f[2 * p + 1]);
}

// Stores vector i of a row.
template <int DT, int TPR, bool kVec>
__device__ __forceinline__ void store_vec(void* base, size_t first, int i, unsigned t, unsigned cols, const float2* x) {
    constexpr int VE = Elem<DT>::kVE, W = PerWord<DT>::kN;
    float f[VE];
#pragma unroll
    for (int p = 0; p < VE / 2; ++p) f[2 * p] = x[p].x, f[2 * p + 1] = x[p].y;
    if (kVec) {
        const unsigned k = i * TPR + t;
        if (k * VE < cols)
            st_stream(reinterpret_cast<uint4*>(static_cast<char*>(base) + first * Elem<DT>::kSize) + k,
                      make_uint4(narrow_word<DT>(f), narrow_word<DT>(f + W), narrow_word<DT>(f + 2 * W),
                                 narrow_word<DT>(f + 3 * W)));
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const unsigned c = (i * VE + e) * TPR + t;
            if (c < cols) store_elem<DT>(base, first + c, f[e]);
        }
    }
}

// Vector i of a parameter (type fp32 or DT; the kVec layout needs it on a
// 16-byte boundary), or `none` where there is no parameter.
template <int DT, int TPR, bool kVec>
__device__ __forceinline__ void load_param(const void* p, bool w32, int i, unsigned t, unsigned cols, float none,
                                           float2* x) {
    constexpr int VE = Elem<DT>::kVE;
    if (p == nullptr) {
#pragma unroll
        for (int e = 0; e < VE / 2; ++e) x[e] = pair(none);
    } else if (kVec) {
        const unsigned k = i * TPR + t;
        if (k * VE >= cols) {
#pragma unroll
            for (int e = 0; e < VE / 2; ++e) x[e] = pair(none);
        } else if (w32) {
            const float4* f = static_cast<const float4*>(p) + k * (VE / 4);
#pragma unroll
            for (int q = 0; q < VE / 4; ++q) {
                const float4 v = f[q];
                x[2 * q] = make_float2(v.x, v.y), x[2 * q + 1] = make_float2(v.z, v.w);
            }
        } else {
            widen<DT>(static_cast<const uint4*>(p)[k], x);
        }
    } else {
        float f[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const unsigned c = (i * VE + e) * TPR + t;
            f[e] = c >= cols ? none : (w32 ? static_cast<const float*>(p)[c] : load_elem<DT>(p, c));
        }
#pragma unroll
        for (int e = 0; e < VE / 2; ++e) x[e] = make_float2(f[2 * e], f[2 * e + 1]);
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

__device__ __forceinline__ float2 shfl_xor2(float2 v, int d) {
    return make_float2(__shfl_xor_sync(0xFFFFFFFFu, v.x, d), __shfl_xor_sync(0xFFFFFFFFu, v.y, d));
}

// Two sums over groups of N lanes.
template <int N> __device__ __forceinline__ float2 lanes_sum2(float2 v) {
#pragma unroll
    for (int d = N / 2; d > 0; d >>= 1) v = __fadd2_rn(v, shfl_xor2(v, d));
    return v;
}

// s / n from the rounded 1 / n, corrected by the remainder.
__device__ __forceinline__ float quotient(float s, float n, float inv_n) {
    const float m = __fmul_rn(s, inv_n);
    return fabsf(m) < __int_as_float(0x7F800000) ? __fmaf_rn(__fmaf_rn(-m, n, s), inv_n, m) : m;
}

// A warp's squares around `mean` from its sum, its squares q around its own m,
// and its number of elements (p = s, q, m, n).
__device__ __forceinline__ float around(const float4& p, float mean) {
    const float d = __fsub_rn(p.z, mean), off = __fmaf_rn(-p.w, p.z, p.x);
    return __fmaf_rn(__fmaf_rn(p.w, d, __fmul_rn(2.0f, off)), d, p.y);
}

// A joined sum of squares; NaN stays (fmaxf would drop it).
__device__ __forceinline__ float not_below_zero(float q) { return q < 0.0f ? 0.0f : q; }

// Backward, a place past a row's end holds x = 0 and dy = 0, which add nothing
// unless (0 - mean) rstd is infinite (a row of great value, all but constant): 0
// times that is NaN, where the row's own h are finite.  For such a row only its
// own places are summed.  (fp16's means are below 2^16 and a finite rstd below
// 2^75.)  The comparison, a row's once, costs rows off 16-byte boundaries 0 to 3%
// (us: 16384 x 1021 bf16 33.1 / 33.1, 8192 x 4099 60.6 / 62.3, 100 x 1021 5.1 /
// 5.2); places masked after the mean is taken off, in every row, cost 4 to 6%.
template <int DT> __device__ __forceinline__ bool past_range(float mean, float rstd) {
    return DT != SAR_FP16 && fabsf(__fmul_rn(mean, rstd)) == __int_as_float(0x7F800000);
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
// which keeps the digits that sum x^2 - n mean^2 would lose.  s_w is rounded, so
// for a row far from zero and all but constant the sum can come out below zero,
// by about what the mean's own rounding is worth: not_below_zero.
// ---------------------------------------------------------------------------
// The parameters are loaded after the statistics, except with kEarly (one vector
// a thread, for calls of few rows, where the loads' latency counts).
template <int TPR, int NV> struct ForwardShape {
    static constexpr int kThreads = TPR < 128 ? 128 : TPR;
    // Resident blocks to compile for: 1024 threads an SM (64 registers).
    static constexpr int kBlocks = NV > 4 ? 1 : 1024 / kThreads;
};

template <int DT, int TPR, int NV, bool kVec, bool kEarly>
__global__ void __launch_bounds__(ForwardShape<TPR, NV>::kThreads, ForwardShape<TPR, NV>::kBlocks)
forward_kernel(NormArgs a, bool w32, float inv_n) {
    constexpr int VE = Elem<DT>::kVE, P = VE / 2, BT = ForwardShape<TPR, NV>::kThreads, RPB = BT / TPR;
    constexpr int WPG = TPR > 32 ? TPR / 32 : 1;
    __shared__ float4 red[TPR > 32 ? WPG : 1];
    const unsigned t = threadIdx.x % TPR, cols = static_cast<unsigned>(a.cols);
    const float n = static_cast<float>(cols);
    pdl_wait();
    float2 we[kEarly ? P : 1], be[kEarly ? P : 1];
    if (kEarly) {
        load_param<DT, TPR, kVec>(a.weight, w32, 0, t, cols, 1.0f, we);
        load_param<DT, TPR, kVec>(a.bias, w32, 0, t, cols, 0.0f, be);
    }
    const size_t groups = static_cast<size_t>(gridDim.x) * RPB;
    // All threads of a block make the same number of rounds.
    for (size_t r0 = static_cast<size_t>(blockIdx.x) * RPB; r0 < a.rows; r0 += groups) {
        const size_t r = r0 + threadIdx.x / TPR;
        const bool live = RPB == 1 || r < a.rows;
        Raw<DT, NV> x;
        load_row<DT, TPR, NV, kVec>(x, a.x, live ? r * a.ldx : 0, t, live ? cols : 0u);
        float2 s2 = pair(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float2 f[P];
            widen<DT>(x.v[i], f);
#pragma unroll
            for (int p = 0; p < P; ++p) s2 = __fadd2_rn(s2, f[p]);
        }
        // Elements of this warp (or group of lanes): whole warps but the last.
        float have = n;
        if (TPR > 32) {
            unsigned k = 0;
#pragma unroll
            for (int i = 0; i < NV * (kVec ? 1 : VE); ++i) {
                const unsigned from = (i * TPR + (t & ~31u)) * (kVec ? VE : 1);
                const unsigned left = from < cols ? cols - from : 0u;
                k += left < 32u * (kVec ? VE : 1) ? left : 32u * (kVec ? VE : 1);
            }
            have = static_cast<float>(k);
        }
        float s = lanes_sum<TPR>(__fadd_rn(s2.x, s2.y));
        // Any value near the warp's mean serves: what it is off is made up for
        // when the warps' parts are joined.
        float mean = TPR > 32 ? __fmul_rn(s, __fdividef(1.0f, fmaxf(have, 1.0f))) : quotient(s, n, inv_n);
        float2 q2 = pair(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float2 f[P];
            widen<DT>(x.v[i], f);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                float2 d = __fadd2_rn(f[p], pair(-mean));
                if (!in_row<DT, TPR, kVec>(i, 2 * p, t, cols)) d.x = 0.0f;
                if (!in_row<DT, TPR, kVec>(i, 2 * p + 1, t, cols)) d.y = 0.0f;
                q2 = __ffma2_rn(d, d, q2);
            }
        }
        float q = lanes_sum<TPR>(__fadd_rn(q2.x, q2.y));
        if (TPR > 32) {
            if ((t & 31) == 0) red[t / 32] = make_float4(s, q, mean, have);
            group_sync<TPR, BT>(0);
            // sum (x - m)^2 = q_w + 2 (m_w - m) (s_w - n_w m_w) + n_w (m_w - m)^2 for a warp.
            if (WPG <= 8) {
                s = 0.0f;
#pragma unroll
                for (int w = 0; w < WPG; ++w) s = __fadd_rn(s, red[w].x);
                mean = quotient(s, n, inv_n);
                q = 0.0f;
#pragma unroll
                for (int w = 0; w < WPG; ++w) q = __fadd_rn(q, around(red[w], mean));
            } else {
                const float4 p = red[(t & 31) % WPG];
                s = p.x;
#pragma unroll
                for (int d = WPG / 2; d > 0; d >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, d));
                mean = quotient(s, n, inv_n);
                q = around(p, mean);
#pragma unroll
                for (int d = WPG / 2; d > 0; d >>= 1) q = __fadd_rn(q, __shfl_xor_sync(0xFFFFFFFFu, q, d));
            }
            q = not_below_zero(q);
        }
        const float rstd = rsqrtf(__fmaf_rn(q, inv_n, a.eps));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float2 f[P], w[P], b[P];
            if (kEarly) {
#pragma unroll
                for (int p = 0; p < P; ++p) w[p] = we[p % (kEarly ? P : 1)], b[p] = be[p % (kEarly ? P : 1)];
            } else {
                load_param<DT, TPR, kVec>(a.weight, w32, i, t, cols, 1.0f, w);
                load_param<DT, TPR, kVec>(a.bias, w32, i, t, cols, 0.0f, b);
            }
            widen<DT>(x.v[i], f);
#pragma unroll
            for (int p = 0; p < P; ++p)
                f[p] = __ffma2_rn(__fmul2_rn(__fadd2_rn(f[p], pair(-mean)), pair(rstd)), w[p], b[p]);
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

template <int DT, int TPR, bool kVec>
__global__ void __launch_bounds__(BackwardShape<TPR>::kThreads, TPR <= 512 ? 2 : 1)
backward_kernel(NormGradArgs a, bool w32, float inv_n) {
    constexpr int VE = Elem<DT>::kVE, P = VE / 2, BT = BackwardShape<TPR>::kThreads, G = BT / TPR;
    constexpr int WPG = TPR > 32 ? TPR / 32 : 1;
    __shared__ float2 red[2][G][WPG];
    extern __shared__ __align__(16) float sums[];                   // [G][TPR * VE], groups of at least a warp
    pdl_wait();
    const unsigned t = threadIdx.x % TPR, cols = static_cast<unsigned>(a.cols);
    const int g = threadIdx.x / TPR;
    const size_t step = static_cast<size_t>(gridDim.x) * G;
    float2 dw[P], db[P];
#pragma unroll
    for (int p = 0; p < P; ++p) dw[p] = db[p] = pair(0.0f);
    Raw<DT, 1> x, dy;
    float mean = 0.0f, rstd = 0.0f;
    // Groups smaller than a warp keep its lanes together: the warp makes the
    // rounds of its first group, lanes without a row on zeros.
    const size_t first = static_cast<size_t>(blockIdx.x) * G;
    size_t r = first + g, lead = first + (TPR < 32 ? (threadIdx.x & ~31u) / TPR : g);
    auto fetch = [&] {
        const bool live = r < a.rows;
        load_row<DT, TPR, 1, kVec>(x, a.x, live ? r * a.ldx : 0, t, live ? cols : 0u);
        load_row<DT, TPR, 1, kVec>(dy, a.dy, live ? r * a.lddy : 0, t, live ? cols : 0u);
        mean = live && (!kVec || t * VE < cols) ? a.mean[r] : 0.0f;        // whole vectors past the end: 0 - 0
        rstd = live ? a.rstd[r] : 0.0f;
    };
    fetch();
    for (int buf = 0; lead < a.rows; lead += step, buf ^= 1) {
        const size_t row = r;
        const float rs = rstd;
        float2 h[P], gr[P], s2 = pair(0.0f), q2 = pair(0.0f);
        {
            float2 d[P], w[P];
            widen<DT>(x.v[0], h);
            widen<DT>(dy.v[0], d);
            const float m = -mean;
            r += step;
            fetch();
            load_param<DT, TPR, kVec>(a.weight, w32, 0, t, cols, 1.0f, w);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                h[p] = __fmul2_rn(__fadd2_rn(h[p], pair(m)), pair(rs));
                gr[p] = __fmul2_rn(d[p], w[p]);
                s2 = __fadd2_rn(s2, gr[p]);
                q2 = __ffma2_rn(gr[p], h[p], q2);
                dw[p] = __ffma2_rn(d[p], h[p], dw[p]);
                db[p] = __fadd2_rn(db[p], d[p]);
            }
            if (!kVec && past_range<DT>(m, rs)) {
                q2 = pair(0.0f);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    if (in_row<DT, TPR, kVec>(0, 2 * p, t, cols)) q2.x = __fmaf_rn(gr[p].x, h[p].x, q2.x);
                    if (in_row<DT, TPR, kVec>(0, 2 * p + 1, t, cols)) q2.y = __fmaf_rn(gr[p].y, h[p].y, q2.y);
                }
            }
        }
        float2 sum = make_float2(__fadd_rn(s2.x, s2.y), __fadd_rn(q2.x, q2.y));
        sum = lanes_sum2<(TPR < 32 ? TPR : 32)>(sum);
        if (TPR > 32) {
            if ((t & 31) == 0) red[buf][g][t / 32] = sum;
            group_sync<TPR, BT>(g);
            sum = lanes_sum2<WPG>(red[buf][g][(t & 31) % WPG]);
        }
        // dx = rstd g - rstd mean(g) - h rstd mean(g h)
        const float c0 = -__fmul_rn(rs, __fmul_rn(sum.x, inv_n)), c1 = -__fmul_rn(rs, __fmul_rn(sum.y, inv_n));
        const bool live = row < a.rows;
#pragma unroll
        for (int p = 0; p < P; ++p) gr[p] = __ffma2_rn(gr[p], pair(rs), __ffma2_rn(h[p], pair(c1), pair(c0)));
        store_vec<DT, TPR, kVec>(a.dx, live ? row * a.lddx : 0, 0, t, live ? cols : 0u, gr);
    }
    if (a.dweight == nullptr && a.dbias == nullptr) return;
    float* out = a.partial + static_cast<size_t>(blockIdx.x) * 2 * cols;
    constexpr int C = TPR * VE, S = TPR < 32 ? BT / 32 : G;
    if (TPR < 32) {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int d = TPR; d < 32; d <<= 1) {
                dw[p] = __fadd2_rn(dw[p], shfl_xor2(dw[p], d));
                db[p] = __fadd2_rn(db[p], shfl_xor2(db[p], d));
            }
    }
    // The groups' sums, added in order; through shared memory, so that they
    // leave in whole sectors.
    const int slot = TPR < 32 ? threadIdx.x / 32 : g;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if (half == 1) __syncthreads();
        if (TPR >= 32 || (threadIdx.x & 31) < TPR) {
            if (kVec) {                               // four columns at a time: single ones would meet in the banks
#pragma unroll
                for (int p = 0; p < P; p += 2) {
                    const float2 u = half == 0 ? dw[p] : db[p], v = half == 0 ? dw[p + 1] : db[p + 1];
                    *reinterpret_cast<float4*>(sums + slot * C + t * VE + 2 * p) = make_float4(u.x, u.y, v.x, v.y);
                }
            } else {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float2 v = half == 0 ? dw[e / 2] : db[e / 2];
                    sums[slot * C + e * TPR + t] = e % 2 ? v.y : v.x;
                }
            }
        }
        __syncthreads();
        for (unsigned c = threadIdx.x; c < cols; c += BT) {
            float v = sums[c];
            for (int p = 1; p < S; ++p) v = __fadd_rn(v, sums[p * C + c]);
            out[half * cols + c] = v;
        }
    }
}

// Threads per row of the backward kernel for a row of `vecs` vectors.
inline int backward_tpr(size_t vecs) {
    int tpr = 8;
    while (tpr < 1024 && static_cast<size_t>(tpr) < vecs) tpr *= 2;
    return tpr;
}

template <int DT> cudaError_t forward(const NormArgs& a, bool w32, bool vec, cudaStream_t s);
template <int DT> cudaError_t backward(const NormGradArgs& a, bool w32, bool vec, unsigned blocks, cudaStream_t s);
// The kernels for many rows (layer_norm_ring.cuh).
constexpr size_t kRingVecs = 2048;
// Vectors per thread, and a block's groups and their warps.
inline int ring_vectors(size_t vecs) { return vecs <= 512 ? 1 : (vecs <= 1024 ? 2 : 4); }
struct RingSplit {
    int groups, warps;
};
inline RingSplit ring_split(size_t vecs, int nv) {
    const int warps = static_cast<int>((vecs + 32 * nv - 1) / (32 * nv)), all = nv == 1 ? 32 : 16;
    const int groups = all / warps;
    return {warps > 1 && groups > 15 ? 15 : groups, warps};        // 15 barriers beside the block's own
}
// Where the rows start: row r is (start + r * step) % (16 / element size)
// elements past a 16-byte boundary, with this period; period 0: every row starts
// on a boundary and is whole vectors long.
struct Alignment {
    unsigned start, step, period;
};
template <int DT> cudaError_t ring_forward(const NormArgs& a, bool w32, size_t vecs, const Alignment& al, cudaStream_t s);
template <int DT> cudaError_t ring_backward(const NormGradArgs& a, bool w32, size_t vecs, const Alignment& al, cudaStream_t s);

template <int DT, int TPR, int NV, bool kEarly = false>
cudaError_t forward_launch(const NormArgs& a, bool w32, bool vec, cudaStream_t s) {
    constexpr int BT = ForwardShape<TPR, NV>::kThreads, RPB = BT / TPR;
    const size_t blocks = (a.rows + RPB - 1) / RPB;
    const dim3 grid(static_cast<unsigned>(blocks < 0x7FFFFFFF ? blocks : 0x7FFFFFFF));
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    return vec ? launch_kernel(forward_kernel<DT, TPR, NV, true, kEarly>, grid, dim3(BT), s, a, w32, inv_n)
               : launch_kernel(forward_kernel<DT, TPR, NV, false, kEarly>, grid, dim3(BT), s, a, w32, inv_n);
}

template <int DT, int TPR>
cudaError_t backward_launch(const NormGradArgs& a, bool w32, bool vec, unsigned blocks, cudaStream_t s) {
    constexpr int BT = BackwardShape<TPR>::kThreads, G = BT / TPR, S = TPR < 32 ? BT / 32 : G;
    const size_t smem = static_cast<size_t>(S) * TPR * Elem<DT>::kVE * sizeof(float);
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    return vec ? launch_kernel_smem(backward_kernel<DT, TPR, true>, dim3(blocks), dim3(BT), smem, s, a, w32, inv_n)
               : launch_kernel_smem(backward_kernel<DT, TPR, false>, dim3(blocks), dim3(BT), smem, s, a, w32, inv_n);
}

// Threads up to which one vector a thread, with its parameters loaded at once, is
// faster: while all rows are on the SMs together.  Measured (us, so / several
// vectors a thread): 8 x 4096 bf16 1.9 / 2.5, 300 x 4096 2.5 / 2.9, 600 x 4096
// 4.2 / 3.3, 1000 x 1024 2.3 / 2.9, 300 x 8192 4.6 / 3.75.
constexpr size_t kEarlyThreads = static_cast<size_t>(kSMs) * 1024;

// Definitions for one element type (layer_norm_<type>.cu).
template <int DT> cudaError_t forward_any(const NormArgs& a, bool w32, bool vec, cudaStream_t s) {
    const size_t vecs = (a.cols + Elem<DT>::kVE - 1) / Elem<DT>::kVE;
    if (vecs > 32 && vecs <= 1024) {
        const size_t tpr = vecs <= 128 ? 128 : (vecs <= 256 ? 256 : (vecs <= 512 ? 512 : 1024));
        if (a.rows * tpr <= kEarlyThreads) {
            if (tpr == 128) return forward_launch<DT, 128, 1, true>(a, w32, vec, s);
            if (tpr == 256) return forward_launch<DT, 256, 1, true>(a, w32, vec, s);
            if (tpr == 512) return forward_launch<DT, 512, 1, true>(a, w32, vec, s);
            return forward_launch<DT, 1024, 1, true>(a, w32, vec, s);
        }
    }
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
    case 8: return backward_launch<DT, 8>(a, w32, vec, blocks, s);
    case 16: return backward_launch<DT, 16>(a, w32, vec, blocks, s);
    case 32: return backward_launch<DT, 32>(a, w32, vec, blocks, s);
    case 64: return backward_launch<DT, 64>(a, w32, vec, blocks, s);
    case 128: return backward_launch<DT, 128>(a, w32, vec, blocks, s);
    case 256: return backward_launch<DT, 256>(a, w32, vec, blocks, s);
    case 512: return backward_launch<DT, 512>(a, w32, vec, blocks, s);
    default: return backward_launch<DT, 1024>(a, w32, vec, blocks, s);
    }
}

}  // namespace norm
}  // namespace sar
