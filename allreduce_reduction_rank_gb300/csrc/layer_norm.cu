// layer_norm.cu -- layer norm and its gradient.
//
// Forward, per row of C elements:  mean = sum x / C,  var = sum (x - mean)^2 / C,
// rstd = 1 / sqrt(var + eps),  y = (x - mean) rstd w + b.  Backward, with
// h = (x - mean) rstd and g = dy w:  dx = rstd (g - mean(g) - h mean(g h)),
// dw = sum over rows of dy h,  db = sum over rows of dy.
//
// Rows that fit a block's registers run the kernels of layer_norm.cuh.  Longer
// ones run those here: one block per row, the row read again for each pass
// (from L2), and the parameters' gradients in a kernel of their own, a thread
// per column over a share of the rows.
#include <algorithm>
#include <initializer_list>

#include "layer_norm_ring.cuh"

namespace sar {
namespace {

// Longest rows in registers, in 16-byte vectors.
constexpr size_t kForwardVecs = 8192, kBackwardVecs = 1024;

// Shares of the rows in the parameters' gradients of longer rows.
constexpr size_t kShares = 64;

// Units of a long row: vectors of 16 bytes where every row starts on a 16-byte
// boundary and is whole vectors long (kVec), single elements otherwise.
template <int DT, bool kVec> struct Unit {
    static constexpr int kN = kVec ? Elem<DT>::kVE : 1;

    static __device__ __forceinline__ void load(const void* base, size_t i, float (&f)[kN]) {
        if constexpr (kVec) {
            const uint4 v = ld_stream_ordered(reinterpret_cast<const uint4*>(static_cast<const char*>(base) + i * Elem<DT>::kSize));
            constexpr int W = PerWord<DT>::kN;
            widen_word<DT>(v.x, f);
            widen_word<DT>(v.y, f + W);
            widen_word<DT>(v.z, f + 2 * W);
            widen_word<DT>(v.w, f + 3 * W);
        } else {
            f[0] = load_elem<DT>(base, i);
        }
    }
    static __device__ __forceinline__ void store(void* base, size_t i, const float (&f)[kN]) {
        if constexpr (kVec) {
            constexpr int W = PerWord<DT>::kN;
            st_stream(reinterpret_cast<uint4*>(static_cast<char*>(base) + i * Elem<DT>::kSize),
                      make_uint4(narrow_word<DT>(f), narrow_word<DT>(f + W), narrow_word<DT>(f + 2 * W),
                                 narrow_word<DT>(f + 3 * W)));
        } else {
            store_elem<DT>(base, i, f[0]);
        }
    }
    // kN values of a parameter from column c on.
    template <int WDT> static __device__ __forceinline__ void param(const void* p, size_t c, float none, float (&f)[kN]) {
#pragma unroll
        for (int e = 0; e < kN; ++e) f[e] = p != nullptr ? load_elem<WDT>(p, c + e) : none;
    }
};

constexpr int kLongThreads = 512;

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
    for (unsigned w = 0; w < kLongThreads / 32; ++w) s = __fadd_rn(s, red[w]);
    return s;
}

template <int DT, int WDT, bool kVec>
__global__ void __launch_bounds__(kLongThreads) long_forward_kernel(NormArgs a) {
    using U = Unit<DT, kVec>;
    constexpr int N = U::kN;
    __shared__ float red[kLongThreads / 32];
    pdl_wait();
    const float n = static_cast<float>(a.cols);
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const size_t bx = r * a.ldx, by = r * a.ldy;
        float s = 0.0f, f[N], w[N], b[N];
        for (size_t c = threadIdx.x * N; c < a.cols; c += kLongThreads * N) {
            U::load(a.x, bx + c, f);
#pragma unroll
            for (int e = 0; e < N; ++e) s = __fadd_rn(s, f[e]);
        }
        const float mean = block_sum(s, red) / n;
        float q = 0.0f;
        for (size_t c = threadIdx.x * N; c < a.cols; c += kLongThreads * N) {
            U::load(a.x, bx + c, f);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float d = __fsub_rn(f[e], mean);
                q = __fmaf_rn(d, d, q);
            }
        }
        const float rstd = 1.0f / sqrtf(block_sum(q, red) / n + a.eps);
        for (size_t c = threadIdx.x * N; c < a.cols; c += kLongThreads * N) {
            U::load(a.x, bx + c, f);
            U::template param<WDT>(a.weight, c, 1.0f, w);
            U::template param<WDT>(a.bias, c, 0.0f, b);
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = __fmaf_rn(__fmul_rn(__fsub_rn(f[e], mean), rstd), w[e], b[e]);
            U::store(a.y, by + c, f);
        }
        if (threadIdx.x == 0) {
            if (a.mean != nullptr) a.mean[r] = mean;
            if (a.rstd != nullptr) a.rstd[r] = rstd;
        }
    }
}

template <int DT, int WDT, bool kVec>
__global__ void __launch_bounds__(kLongThreads) long_dx_kernel(NormGradArgs a) {
    using U = Unit<DT, kVec>;
    constexpr int N = U::kN;
    __shared__ float red[kLongThreads / 32];
    pdl_wait();
    const float n = static_cast<float>(a.cols);
    for (size_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const size_t bx = r * a.ldx, bd = r * a.lddy, bo = r * a.lddx;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s = 0.0f, q = 0.0f, x[N], d[N], w[N];
        for (size_t c = threadIdx.x * N; c < a.cols; c += kLongThreads * N) {
            U::load(a.x, bx + c, x);
            U::load(a.dy, bd + c, d);
            U::template param<WDT>(a.weight, c, 1.0f, w);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float h = __fmul_rn(__fsub_rn(x[e], mean), rstd), g = __fmul_rn(d[e], w[e]);
                s = __fadd_rn(s, g);
                q = __fmaf_rn(g, h, q);
            }
        }
        const float mg = block_sum(s, red) / n, mgh = block_sum(q, red) / n;
        for (size_t c = threadIdx.x * N; c < a.cols; c += kLongThreads * N) {
            U::load(a.x, bx + c, x);
            U::load(a.dy, bd + c, d);
            U::template param<WDT>(a.weight, c, 1.0f, w);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float h = __fmul_rn(__fsub_rn(x[e], mean), rstd), g = __fmul_rn(d[e], w[e]);
                x[e] = __fmul_rn(rstd, __fmaf_rn(-h, mgh, __fsub_rn(g, mg)));
            }
            U::store(a.dx, bo + c, x);
        }
    }
}

// Sums of dy h and dy over a share of the rows, a thread per unit of columns.
template <int DT, bool kVec>
__global__ void __launch_bounds__(kThreads) long_shares_kernel(NormGradArgs a) {
    using U = Unit<DT, kVec>;
    constexpr int N = U::kN;
    pdl_wait();
    const size_t shares = gridDim.y, per = (a.rows + shares - 1) / shares;
    const size_t r0 = per * blockIdx.y, r1 = r0 + per < a.rows ? r0 + per : a.rows;
    for (size_t c = (static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x) * N; c < a.cols;
         c += static_cast<size_t>(gridDim.x) * kThreads * N) {
        float w[N], b[N];
#pragma unroll
        for (int e = 0; e < N; ++e) w[e] = b[e] = 0.0f;
#pragma unroll 2
        for (size_t r = r0; r < r1; ++r) {
            float x[N], d[N];
            U::load(a.x, r * a.ldx + c, x);
            U::load(a.dy, r * a.lddy + c, d);
            const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                w[e] = __fmaf_rn(d[e], __fmul_rn(__fsub_rn(x[e], mean), rstd), w[e]);
                b[e] = __fadd_rn(b[e], d[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            a.partial[blockIdx.y * 2 * a.cols + c + e] = w[e];
            a.partial[(blockIdx.y * 2 + 1) * a.cols + c + e] = b[e];
        }
    }
}

// dweight and dbias from the shares' sums: a warp reads 32 * N columns of a share
// (N = 4, as float4, where the columns allow it), a block's warps have every
// kParamWarps-th share, ten loads in flight, and are then added in order.
constexpr int kParamWarps = 16;
template <int WDT, int N>
__global__ void __launch_bounds__(kParamWarps * 32) params_kernel(NormGradArgs a, unsigned shares) {
    __shared__ float part[kParamWarps][32 * N];
    pdl_wait();
    const unsigned lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool bias = blockIdx.y != 0;
    void* out = bias ? a.dbias : a.dweight;
    if (out == nullptr) return;
    for (size_t c0 = static_cast<size_t>(blockIdx.x) * 32 * N; c0 < a.cols; c0 += static_cast<size_t>(gridDim.x) * 32 * N) {
        const size_t c = c0 + lane * N;
        float v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = 0.0f;
        if (c < a.cols) {
            for (unsigned k0 = warp; k0 < shares; k0 += 10 * kParamWarps) {
                float p[10][N];
#pragma unroll
                for (int i = 0; i < 10; ++i) {
                    const unsigned k = k0 + i * kParamWarps;
                    const float* from = a.partial + (static_cast<size_t>(k) * 2 + bias) * a.cols + c;
                    if constexpr (N == 4) {
                        const float4 f = k < shares ? *reinterpret_cast<const float4*>(from) : make_float4(0, 0, 0, 0);
                        p[i][0] = f.x, p[i][1] = f.y, p[i][2] = f.z, p[i][3] = f.w;
                    } else {
                        p[i][0] = k < shares ? *from : 0.0f;
                    }
                }
#pragma unroll
                for (int i = 0; i < 10; ++i)
#pragma unroll
                    for (int e = 0; e < N; ++e) v[e] = __fadd_rn(v[e], p[i][e]);
            }
        }
#pragma unroll
        for (int e = 0; e < N; ++e) part[warp][lane * N + e] = v[e];
        __syncthreads();
        if (threadIdx.x < 32 * N && c0 + threadIdx.x < a.cols) {
            float sum = part[0][threadIdx.x];
            for (int w = 1; w < kParamWarps; ++w) sum = __fadd_rn(sum, part[w][threadIdx.x]);
            store_elem<WDT>(out, c0 + threadIdx.x, sum);
        }
        __syncthreads();
    }
}

template <int WDT, int N> cudaError_t params_launch(const NormGradArgs& a, unsigned shares, cudaStream_t s) {
    const size_t blocks = (a.cols + 32 * N - 1) / (32 * N);
    return launch_kernel(params_kernel<WDT, N>, dim3(static_cast<unsigned>(blocks < 65535 ? blocks : 65535), 2),
                         dim3(kParamWarps * 32), s, a, shares);
}

template <int WDT> cudaError_t params(const NormGradArgs& a, unsigned shares, cudaStream_t s) {
    return a.cols % 4 == 0 && a.cols >= 4096 ? params_launch<WDT, 4>(a, shares, s) : params_launch<WDT, 1>(a, shares, s);
}

cudaError_t params_of(sar_dtype wdt, const NormGradArgs& a, unsigned shares, cudaStream_t s) {
    switch (wdt) {
    case SAR_BF16: return params<SAR_BF16>(a, shares, s);
    case SAR_FP16: return params<SAR_FP16>(a, shares, s);
    default: return params<SAR_FP32>(a, shares, s);
    }
}

unsigned blocks_for(size_t items, size_t per, size_t cap) {
    const size_t g = (items + per - 1) / per;
    return static_cast<unsigned>(g < 1 ? 1 : (g > cap ? cap : g));
}

template <int DT, int WDT> cudaError_t long_forward(const NormArgs& a, bool vec, cudaStream_t s) {
    const dim3 grid(blocks_for(a.rows, 1, 1u << 30)), block(kLongThreads);
    return vec ? launch_kernel(long_forward_kernel<DT, WDT, true>, grid, block, s, a)
               : launch_kernel(long_forward_kernel<DT, WDT, false>, grid, block, s, a);
}

template <int DT, int WDT> cudaError_t long_backward(const NormGradArgs& a, unsigned shares, bool vec, cudaStream_t s) {
    if (a.dweight != nullptr || a.dbias != nullptr) {
        const size_t per = kThreads * (vec ? Elem<DT>::kVE : 1);
        const dim3 grid(blocks_for(a.cols, per, 65535), shares), block(kThreads);
        const cudaError_t e = vec ? launch_kernel(long_shares_kernel<DT, true>, grid, block, s, a)
                                  : launch_kernel(long_shares_kernel<DT, false>, grid, block, s, a);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid(blocks_for(a.rows, 1, 1u << 30)), block(kLongThreads);
    return vec ? launch_kernel(long_dx_kernel<DT, WDT, true>, grid, block, s, a)
               : launch_kernel(long_dx_kernel<DT, WDT, false>, grid, block, s, a);
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows of `cols` elements of `es` bytes move as whole 16-byte vectors.
bool rows_on16(const void* p, size_t ld, size_t rows, size_t es) { return on16(p) && (rows <= 1 || ld * es % 16 == 0); }

// Rows for a group of the ring kernels' blocks from which they are faster than
// the kernels of layer_norm.cuh, with one vector a thread: the ring fills for 3
// us before it pays.  `odd`: 16-bit rows at odd alignments, whose other kernel
// moves single elements.  Measured (us, other kernel / ring): forward 1900 x
// 4096 bf16 (6 rows a group) 8.8 / 9.4, 2600 x 4096 (9) 11.4 / 11.4, 2600 x 1021
// bf16 (3) 10.2 / 6.7; backward 1300 x 4096 fp16 (4) 13.3 / 13.6, 1900 x 4096
// bf16 (6) 16.7 / 15.4, 4099 x 1021 fp32 (7) 15.4 / 13.9, 6000 x 1021 bf16 (7)
// 16.3 / 17.9.  With more vectors a thread 2 is enough (650 x 8192 bf16, 4 rows:
// 8.0 / 7.0, backward 14.4 / 12.8).
struct Least {
    size_t whole, odd;
};
constexpr Least kForwardLeast = {8, 2}, kBackwardLeast = {5, 8};

// A matrix of a call to the kernels for many rows.
struct Matrix {
    const void* p;
    size_t ld;
};

// Whether those kernels take the call: rows that they hold, enough for every
// group of their blocks, and matrices whose rows start alike.
bool ring_takes(std::initializer_list<Matrix> all, size_t rows, size_t cols, size_t es, const Least& least, size_t* vecs,
                norm::Alignment* al) {
    const size_t ve = 16 / es;
    const Matrix& m = *all.begin();
    const size_t start = reinterpret_cast<uintptr_t>(m.p) / es % ve, step = m.ld % ve;
    for (const Matrix& o : all)
        if (reinterpret_cast<uintptr_t>(o.p) / es % ve != start || o.ld % ve != step) return false;
    size_t most = 0, period = 1;                      // largest shift, rows until it repeats
    if (start != 0 || step != 0) {
        while (period * step % ve != 0) period *= 2;
        for (size_t r = 0; r < period; ++r) most = std::max(most, (start + r * step) % ve);
    }
    const bool whole = start == 0 && step == 0 && cols % ve == 0;
    *vecs = (cols + most + ve - 1) / ve;
    *al = {static_cast<unsigned>(start), static_cast<unsigned>(step), static_cast<unsigned>(whole ? 0 : period)};
    if (*vecs <= 16 || *vecs > norm::kRingVecs || rows > 0x7FFFFFFF) return false;
    const int nv = norm::ring_vectors(*vecs);
    const size_t many = nv > 1 ? 2 : (whole || es != 2 ? least.whole : least.odd);
    return rows >= many * norm::kSMs * norm::ring_split(*vecs, nv).groups;
}

template <int DT> cudaError_t forward_of(sar_dtype wdt, const NormArgs& a, cudaStream_t s) {
    constexpr size_t es = Elem<DT>::kSize, VE = Elem<DT>::kVE;
    size_t vecs;
    norm::Alignment al;
    if (ring_takes({{a.x, a.ldx}, {a.y, a.ldy}}, a.rows, a.cols, es, kForwardLeast, &vecs, &al))
        return norm::ring_forward<DT>(a, wdt == SAR_FP32, vecs, al, s);
    const bool rows16 = a.cols % VE == 0 && rows_on16(a.x, a.ldx, a.rows, es) && rows_on16(a.y, a.ldy, a.rows, es);
    if ((a.cols + VE - 1) / VE > kForwardVecs)
        return wdt == SAR_FP32 ? long_forward<DT, SAR_FP32>(a, rows16, s) : long_forward<DT, DT>(a, rows16, s);
    const bool vec = rows16 && on16(a.weight) && on16(a.bias);
    return norm::forward<DT>(a, wdt == SAR_FP32, vec, s);
}

// Blocks of the register kernel: enough groups for the rows (two rows each where
// the parameters' gradients are wanted, since each block leaves a row of sums),
// at most what the SMs hold at a time.
template <int DT> unsigned backward_blocks(size_t rows, size_t cols, bool params) {
    const int tpr = norm::backward_tpr((cols + Elem<DT>::kVE - 1) / Elem<DT>::kVE);
    const int groups = tpr > 512 ? 1 : 512 / tpr;
    const size_t per = params ? 2 * groups : groups, need = (rows + per - 1) / per, fit = tpr > 512 ? norm::kSMs : 2 * norm::kSMs;
    return static_cast<unsigned>(need < fit ? need : fit);
}

template <int DT> cudaError_t backward_of(sar_dtype wdt, const NormGradArgs& a, cudaStream_t s) {
    constexpr size_t es = Elem<DT>::kSize, VE = Elem<DT>::kVE;
    const bool rows16 = a.cols % VE == 0 && rows_on16(a.x, a.ldx, a.rows, es) && rows_on16(a.dy, a.lddy, a.rows, es) &&
                        rows_on16(a.dx, a.lddx, a.rows, es);
    unsigned shares = 0;
    cudaError_t e = cudaSuccess;
    size_t vecs;
    norm::Alignment al;
    if (ring_takes({{a.x, a.ldx}, {a.dy, a.lddy}, {a.dx, a.lddx}}, a.rows, a.cols, es, kBackwardLeast, &vecs, &al)) {
        shares = norm::kSMs;
        e = norm::ring_backward<DT>(a, wdt == SAR_FP32, vecs, al, s);
    } else if (a.rows != 0 && (a.cols + VE - 1) / VE > kBackwardVecs) {
        shares = static_cast<unsigned>(a.rows < kShares ? a.rows : kShares);
        e = wdt == SAR_FP32 ? long_backward<DT, SAR_FP32>(a, shares, rows16, s) : long_backward<DT, DT>(a, shares, rows16, s);
    } else if (a.rows != 0) {
        const bool vec = rows16 && on16(a.weight);
        shares = backward_blocks<DT>(a.rows, a.cols, a.dweight != nullptr || a.dbias != nullptr);
        e = norm::backward<DT>(a, wdt == SAR_FP32, vec, shares, s);
    }
    if (e != cudaSuccess || (a.dweight == nullptr && a.dbias == nullptr)) return e;
    return params_of(wdt, a, shares, s);
}

}  // namespace

// Rows of sums in the workspace: the most that any element type writes.
size_t layer_norm_partials(size_t rows, size_t) {
    const size_t most = 2 * norm::kSMs;
    return rows < 1 ? 1 : (rows < most ? rows : most);
}

cudaError_t launch_layer_norm(sar_dtype dt, sar_dtype wdt, const NormArgs& a, cudaStream_t s) {
    switch (dt) {
    case SAR_BF16: return forward_of<SAR_BF16>(wdt, a, s);
    case SAR_FP16: return forward_of<SAR_FP16>(wdt, a, s);
    case SAR_FP32: return forward_of<SAR_FP32>(wdt, a, s);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_layer_norm_backward(sar_dtype dt, sar_dtype wdt, const NormGradArgs& a, cudaStream_t s) {
    switch (dt) {
    case SAR_BF16: return backward_of<SAR_BF16>(wdt, a, s);
    case SAR_FP16: return backward_of<SAR_FP16>(wdt, a, s);
    case SAR_FP32: return backward_of<SAR_FP32>(wdt, a, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace sar
