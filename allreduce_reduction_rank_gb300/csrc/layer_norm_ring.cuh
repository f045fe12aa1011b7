// layer_norm_ring.cuh -- the layer norm kernels for many rows.
//
// One block of 512 threads per SM stays for many rows.  A row belongs to a
// group of TPR threads, which has a contiguous range of the rows and works on R
// of them at a time (a batch).  Thread t has NV vectors of four 32-bit words of
// each row; it copies them into its own places of a ring of D batches in
// shared memory with cp.async, D - 1 batches ahead, and only itself reads them
// again.  So the copies need no barrier, 100 KB and more are in flight on each
// SM whatever the registers hold, and the parameters and the sums for their
// gradients stay in registers.  What a batch costs beside its elements, the
// sums over the threads and a barrier, is shared by its rows: the sums of R
// rows travel together, halving their number with each exchange between lanes.
//
// W, the bytes of one access, is 16 or 4: word q of thread t is word
// ((q / 4) * TPR + t) * 4 + q % 4 of the row, or word q * TPR + t.
#pragma once

#include "layer_norm.cuh"

namespace sar {
namespace norm {

constexpr int kRingThreads = 512;

template <int W, int TPR> __device__ __forceinline__ unsigned word_of(int q, unsigned t) {
    return W == 16 ? ((q / 4) * TPR + t) * 4 + q % 4 : q * TPR + t;
}

// cp.async of W bytes, or W zero bytes where `have` is false.
template <int W> __device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool have) {
    const int n = have ? W : 0;
    if (W == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A thread's part of one row: NV slots of 16 bytes, the slots of the block's
// threads side by side.
template <int W, int TPR, int NV>
__device__ __forceinline__ void copy_row(uint4* slots, const void* base, size_t byte, unsigned t, unsigned words) {
    const char* row = static_cast<const char*>(base) + byte;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        uint4* slot = slots + i * kRingThreads;
        if (W == 16) {
            const unsigned w = word_of<W, TPR>(4 * i, t);
            copy_async<W>(static_cast<uint32_t>(__cvta_generic_to_shared(slot + threadIdx.x)), row + (w < words ? w * 4 : 0),
                          w < words);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const unsigned w = word_of<W, TPR>(4 * i + k, t);
                copy_async<W>(static_cast<uint32_t>(__cvta_generic_to_shared(
                                  reinterpret_cast<uint32_t*>(slot) + k * kRingThreads + threadIdx.x)),
                              row + (w < words ? w * 4 : 0), w < words);
            }
        }
    }
}

template <int W> __device__ __forceinline__ uint4 read_slot(const uint4* slot) {
    if (W == 16) return slot[threadIdx.x];
    const uint32_t* p = reinterpret_cast<const uint32_t*>(slot) + threadIdx.x;
    return make_uint4(p[0], p[kRingThreads], p[2 * kRingThreads], p[3 * kRingThreads]);
}

// Vector i of a row, stored.
template <int DT, int W, int TPR>
__device__ __forceinline__ void write_vec(void* base, size_t byte, int i, unsigned t, unsigned words, const float2* x) {
    constexpr int VE = Elem<DT>::kVE, N = PerWord<DT>::kN;
    float f[VE];
#pragma unroll
    for (int p = 0; p < VE / 2; ++p) f[2 * p] = x[p].x, f[2 * p + 1] = x[p].y;
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = narrow_word<DT>(f + k * N);
    char* row = static_cast<char*>(base) + byte;
    if (W == 16) {
        const unsigned w = word_of<W, TPR>(4 * i, t);
        if (w < words) st_stream(reinterpret_cast<uint4*>(row + w * 4), make_uint4(u[0], u[1], u[2], u[3]));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const unsigned w = word_of<W, TPR>(4 * i + k, t);
            if (w < words)
                asm volatile("st.global.L1::no_allocate.u32 [%0], %1;" ::"l"(row + w * 4), "r"(u[k]) : "memory");
        }
    }
}

// Column of value v (of VE * NV) of thread t.
template <int DT, int W, int TPR> __device__ __forceinline__ unsigned column_of(int v, unsigned t) {
    constexpr int N = PerWord<DT>::kN;
    return word_of<W, TPR>(v / N, t) * N + v % N;
}

// A thread's values of a parameter of type fp32 or DT; `none` without one.
template <int DT, int W, int TPR, int NV>
__device__ __forceinline__ void read_param(const void* p, bool w32, unsigned t, unsigned cols, float none, float2* x) {
#pragma unroll
    for (int k = 0; k < NV * Elem<DT>::kVE / 2; ++k) {
        const unsigned c0 = column_of<DT, W, TPR>(2 * k, t), c1 = column_of<DT, W, TPR>(2 * k + 1, t);
        x[k] = pair(none);
        if (p != nullptr && c0 < cols) x[k].x = w32 ? static_cast<const float*>(p)[c0] : load_elem<DT>(p, c0);
        if (p != nullptr && c1 < cols) x[k].y = w32 ? static_cast<const float*>(p)[c1] : load_elem<DT>(p, c1);
    }
}

// Sums N values (a power of two) over a warp: value i ends in the lanes
// i * (32 / N) .. + 32 / N - 1.
template <int N> __device__ __forceinline__ float scatter_sum(float (&v)[N]) {
    const unsigned lane = threadIdx.x & 31;
    int bit = 16;
#pragma unroll
    for (int m = N / 2; m > 0; m >>= 1, bit >>= 1) {
        const bool high = lane & bit;
#pragma unroll
        for (int i = 0; i < m; ++i) {
            const float send = high ? v[i] : v[i + m], keep = high ? v[i + m] : v[i];
            v[i] = __fadd_rn(keep, __shfl_xor_sync(0xFFFFFFFFu, send, bit));
        }
    }
    float s = v[0];
    for (; bit > 0; bit >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, bit));
    return s;
}

// The rows of group `g` of `n` in all: contiguous, sizes that differ by at most one.
__device__ __forceinline__ size_t range_start(size_t rows, size_t g, size_t n) {
    const size_t per = rows / n, more = rows % n;
    return per * g + (g < more ? g : more);
}

template <int DT, int W, int TPR, int NV, int R, int D>
__global__ void __launch_bounds__(kRingThreads, 1) ring_forward_kernel(NormArgs a, bool w32, float inv_n) {
    constexpr int VE = Elem<DT>::kVE, P = VE / 2, G = kRingThreads / TPR, WPG = TPR / 32, L = 32 / R;
    constexpr size_t es = Elem<DT>::kSize;
    extern __shared__ uint4 ring[];                   // [D][R][NV][threads]
    __shared__ float4 red[2][kRingThreads / 32][R];
    const unsigned t = threadIdx.x % TPR, cols = static_cast<unsigned>(a.cols), words = cols * es / 4;
    const unsigned lane = threadIdx.x & 31;
    const int g = threadIdx.x / TPR;
    const float n = static_cast<float>(cols);
    pdl_wait();
    const size_t groups = static_cast<size_t>(gridDim.x) * G, id = static_cast<size_t>(blockIdx.x) * G + g;
    const size_t begin = range_start(a.rows, id, groups), end = range_start(a.rows, id + 1, groups);
    size_t ahead = begin;                             // first row of the next batch to copy
    int slot = 0;                                     // its place in the ring
    auto copy_batch = [&] {
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (ahead + j < end)
                copy_row<W, TPR, NV>(ring + (slot * R + j) * NV * kRingThreads, a.x, (ahead + j) * a.ldx * es, t, words);
        copy_commit();
        ahead += R;
        slot = slot + 1 == D ? 0 : slot + 1;
    };
#pragma unroll
    for (int d = 0; d < D - 1; ++d) copy_batch();
    float2 w[NV * P], b[NV * P];
    read_param<DT, W, TPR, NV>(a.weight, w32, t, cols, 1.0f, w);
    read_param<DT, W, TPR, NV>(a.bias, w32, t, cols, 0.0f, b);
    // Elements of this warp.
    unsigned held = 0;
#pragma unroll
    for (int v = 0; v < NV * 4; ++v) held += __popc(__ballot_sync(0xFFFFFFFFu, word_of<W, TPR>(v, t) < words));
    const float have = static_cast<float>(held * PerWord<DT>::kN);
    const float inv_have = have > 0.0f ? 1.0f / have : 0.0f;
    int at = 0;
    for (size_t r = begin, k = 0; r < end; r += R, ++k) {
        copy_wait<D - 2>();
        uint4 x[R][NV];
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < NV; ++i) x[j][i] = read_slot<W>(ring + ((at * R + j) * NV + i) * kRingThreads);
        at = at + 1 == D ? 0 : at + 1;
        copy_batch();
        float s[R], m[R], q[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float2 s2 = pair(0.0f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 f[P];
                widen<DT>(x[j][i], f);
#pragma unroll
                for (int p = 0; p < P; ++p) s2 = __fadd2_rn(s2, f[p]);
            }
            s[j] = __fadd_rn(s2.x, s2.y);
        }
        const float total = scatter_sum<R>(s);
        const float near = __fmul_rn(total, inv_have);
#pragma unroll
        for (int j = 0; j < R; ++j) m[j] = __shfl_sync(0xFFFFFFFFu, near, j * L);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float2 q2 = pair(0.0f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 f[P];
                widen<DT>(x[j][i], f);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    float2 d = __fadd2_rn(f[p], pair(-m[j]));
                    constexpr int N = PerWord<DT>::kN;
                    if (word_of<W, TPR>(4 * i + 2 * p / N, t) >= words) d.x = 0.0f;
                    if (word_of<W, TPR>(4 * i + (2 * p + 1) / N, t) >= words) d.y = 0.0f;
                    q2 = __ffma2_rn(d, d, q2);
                }
            }
            q[j] = __fadd_rn(q2.x, q2.y);
        }
        const float squares = scatter_sum<R>(q);
        float mean, rstd;                             // of row lane % R (TPR > 32), or lane / L
        if (TPR == 32) {
            mean = quotient(total, n, inv_n);
            const float4 p = make_float4(total, squares, near, have);
            rstd = rsqrtf(__fmaf_rn(around(p, mean), inv_n, a.eps));
        } else {
            float4(&all)[kRingThreads / 32][R] = red[k & 1];
            if (lane % L == 0) all[threadIdx.x / 32][lane / L] = make_float4(total, squares, near, have);
            group_sync<TPR, kRingThreads>(g);
            constexpr int T = (WPG + L - 1) / L;      // a lane's warps: lane / R, + L, ...
            float4 p[T];
            float sum = 0.0f, sq = 0.0f;
#pragma unroll
            for (int i = 0; i < T; ++i) {
                const unsigned from = lane / R + i * L;
                p[i] = from < WPG ? all[g * WPG + from][lane % R] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                sum = __fadd_rn(sum, p[i].x);
            }
#pragma unroll
            for (int d = R; d < 32; d <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xFFFFFFFFu, sum, d));
            mean = quotient(sum, n, inv_n);
#pragma unroll
            for (int i = 0; i < T; ++i) sq = __fadd_rn(sq, around(p[i], mean));
#pragma unroll
            for (int d = R; d < 32; d <<= 1) sq = __fadd_rn(sq, __shfl_xor_sync(0xFFFFFFFFu, sq, d));
            rstd = rsqrtf(__fmaf_rn(sq, inv_n, a.eps));
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const float mj = __shfl_sync(0xFFFFFFFFu, mean, TPR == 32 ? j * L : j);
            const float rj = __shfl_sync(0xFFFFFFFFu, rstd, TPR == 32 ? j * L : j);
            if (r + j >= end) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 f[P];
                widen<DT>(x[j][i], f);
#pragma unroll
                for (int p = 0; p < P; ++p)
                    f[p] = __ffma2_rn(__fmul2_rn(__fadd2_rn(f[p], pair(-mj)), pair(rj)), w[i * P + p], b[i * P + p]);
                write_vec<DT, W, TPR>(a.y, (r + j) * a.ldy * es, i, t, words, f);
            }
            if (t == 0) {
                if (a.mean != nullptr) a.mean[r + j] = mj;
                if (a.rstd != nullptr) a.rstd[r + j] = rj;
            }
        }
    }
    copy_wait<0>();
}

// The sums over a group of 2 R values per thread, in every thread of it.
template <int TPR, int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float (*red)[N], int g) {
    constexpr int WPG = TPR / 32, L = 32 / N;
    const unsigned lane = threadIdx.x & 31;
    float s = scatter_sum<N>(v);
    if (TPR == 32) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, s, i * L);
        return;
    }
    if (lane % L == 0) red[threadIdx.x / 32][lane / L] = s;
    group_sync<TPR, kRingThreads>(g);
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < (WPG + L - 1) / L; ++i) {
        const unsigned from = lane / N + i * L;
        if (from < WPG) s = __fadd_rn(s, red[g * WPG + from][lane % N]);
    }
#pragma unroll
    for (int d = N; d < 32; d <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, d));
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, s, i);
}

template <int DT, int W, int TPR, int NV, int R, int D>
__global__ void __launch_bounds__(kRingThreads, 1) ring_backward_kernel(NormGradArgs a, bool w32, float inv_n) {
    constexpr int VE = Elem<DT>::kVE, P = VE / 2, G = kRingThreads / TPR;
    constexpr size_t es = Elem<DT>::kSize;
    // h and g of a batch are kept for dx where the registers hold them, else
    // computed again from the ring.
    constexpr bool kHold = VE == 4 && NV == 1 && W == 16;
    constexpr int HP = kHold ? P : 1;
    extern __shared__ uint4 ring[];                   // [D][R][x, dy][NV][threads]
    __shared__ float red[2][kRingThreads / 32][2 * R];
    const unsigned t = threadIdx.x % TPR, cols = static_cast<unsigned>(a.cols), words = cols * es / 4;
    const int g = threadIdx.x / TPR;
    pdl_wait();
    const size_t groups = static_cast<size_t>(gridDim.x) * G, id = static_cast<size_t>(blockIdx.x) * G + g;
    const size_t begin = range_start(a.rows, id, groups), end = range_start(a.rows, id + 1, groups);
    size_t ahead = begin;
    int slot = 0;
    auto copy_batch = [&] {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (ahead + j >= end) continue;
            uint4* to = ring + (slot * R + j) * 2 * NV * kRingThreads;
            copy_row<W, TPR, NV>(to, a.x, (ahead + j) * a.ldx * es, t, words);
            copy_row<W, TPR, NV>(to + NV * kRingThreads, a.dy, (ahead + j) * a.lddy * es, t, words);
        }
        copy_commit();
        ahead += R;
        slot = slot + 1 == D ? 0 : slot + 1;
    };
#pragma unroll
    for (int d = 0; d < D - 1; ++d) copy_batch();
    float2 w[NV * P], dw[NV * P], db[NV * P];
    read_param<DT, W, TPR, NV>(a.weight, w32, t, cols, 1.0f, w);
#pragma unroll
    for (int p = 0; p < NV * P; ++p) dw[p] = db[p] = pair(0.0f);
    float mean[R], rstd[R];
    auto statistics = [&](size_t r) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            mean[j] = r + j < end ? a.mean[r + j] : 0.0f;
            rstd[j] = r + j < end ? a.rstd[r + j] : 0.0f;
        }
    };
    statistics(begin);
    int at = 0;
    for (size_t r = begin, k = 0; r < end; r += R, ++k) {
        copy_wait<D - 2>();
        copy_batch();                                 // into the place of the batch before this one
        const uint4* from = ring + at * R * 2 * NV * kRingThreads;
        at = at + 1 == D ? 0 : at + 1;
        float v[2 * R], rs[R], mj[R];
        float2 h[R][HP], gr[R][HP];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float2 s2 = pair(0.0f), q2 = pair(0.0f);
            rs[j] = rstd[j], mj[j] = -mean[j];
            if (r + j < end) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float2 f[P], d[P];
                    widen<DT>(read_slot<W>(from + (j * 2 * NV + i) * kRingThreads), f);
                    widen<DT>(read_slot<W>(from + (j * 2 * NV + NV + i) * kRingThreads), d);
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const int c = i * P + p;
                        f[p] = __fmul2_rn(__fadd2_rn(f[p], pair(mj[j])), pair(rs[j]));
                        dw[c] = __ffma2_rn(d[p], f[p], dw[c]);
                        db[c] = __fadd2_rn(db[c], d[p]);
                        d[p] = __fmul2_rn(d[p], w[c]);
                        s2 = __fadd2_rn(s2, d[p]);
                        q2 = __ffma2_rn(d[p], f[p], q2);
                        if (kHold) h[j][p % HP] = f[p], gr[j][p % HP] = d[p];
                    }
                }
            }
            v[2 * j] = __fadd_rn(s2.x, s2.y);
            v[2 * j + 1] = __fadd_rn(q2.x, q2.y);
        }
        statistics(r + R);
        group_sums<TPR, 2 * R>(v, red[k & 1], g);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (r + j >= end) continue;
            // dx = rstd g - rstd mean(g) - h rstd mean(g h)
            const float c0 = -__fmul_rn(rs[j], __fmul_rn(v[2 * j], inv_n)), c1 = -__fmul_rn(rs[j], __fmul_rn(v[2 * j + 1], inv_n));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 f[P], d[P];
                if (kHold) {
#pragma unroll
                    for (int p = 0; p < P; ++p) f[p] = h[j][p % HP], d[p] = gr[j][p % HP];
                } else {
                    widen<DT>(read_slot<W>(from + (j * 2 * NV + i) * kRingThreads), f);
                    widen<DT>(read_slot<W>(from + (j * 2 * NV + NV + i) * kRingThreads), d);
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        f[p] = __fmul2_rn(__fadd2_rn(f[p], pair(mj[j])), pair(rs[j]));
                        d[p] = __fmul2_rn(d[p], w[i * P + p]);
                    }
                }
#pragma unroll
                for (int p = 0; p < P; ++p) f[p] = __ffma2_rn(d[p], pair(rs[j]), __ffma2_rn(f[p], pair(c1), pair(c0)));
                write_vec<DT, W, TPR>(a.dx, (r + j) * a.lddx * es, i, t, words, f);
            }
        }
    }
    copy_wait<0>();
    if (a.dweight == nullptr && a.dbias == nullptr) return;
    float* out = a.partial + static_cast<size_t>(blockIdx.x) * 2 * cols;
    if (G == 1) {
#pragma unroll
        for (int e = 0; e < NV * VE; ++e) {
            const unsigned c = column_of<DT, W, TPR>(e, t);
            if (c < cols) {
                out[c] = e % 2 ? dw[e / 2].y : dw[e / 2].x;
                out[cols + c] = e % 2 ? db[e / 2].y : db[e / 2].x;
            }
        }
        return;
    }
    // The groups' sums, added in order.
    constexpr int C = TPR * NV * VE;
    float* sums = reinterpret_cast<float*>(ring);     // [G][2][C]
    __syncthreads();
#pragma unroll
    for (int e = 0; e < NV * VE; ++e) {
        const unsigned c = column_of<DT, W, TPR>(e, t);
        sums[g * 2 * C + c] = e % 2 ? dw[e / 2].y : dw[e / 2].x;
        sums[(g * 2 + 1) * C + c] = e % 2 ? db[e / 2].y : db[e / 2].x;
    }
    __syncthreads();
    for (unsigned c = threadIdx.x; c < 2 * cols; c += kRingThreads) {
        const unsigned half = c >= cols, k = half * C + (c - half * cols);
        float v = sums[k];
        for (int p = 1; p < G; ++p) v = __fadd_rn(v, sums[p * 2 * C + k]);
        out[c] = v;
    }
}

// Dynamic shared memory above 48 KiB is allowed explicitly, once per device and
// kernel (only a successful call is remembered).
template <class Kernel> cudaError_t allow_smem(Kernel kernel, size_t bytes, std::atomic<bool>* allowed) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!allowed[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
        if (e != cudaSuccess) return e;
        allowed[dev].store(true, std::memory_order_release);
    }
    return cudaSuccess;
}

template <int DT, int W, int TPR, int NV, int R, int D> cudaError_t ring_forward_launch(const NormArgs& a, bool w32, cudaStream_t s) {
    static std::atomic<bool> allowed[kMaxDevices];
    constexpr size_t smem = static_cast<size_t>(D) * R * NV * kRingThreads * 16;
    const cudaError_t e = allow_smem(ring_forward_kernel<DT, W, TPR, NV, R, D>, smem, allowed);
    if (e != cudaSuccess) return e;
    return launch_kernel_smem(ring_forward_kernel<DT, W, TPR, NV, R, D>, dim3(kSMs), dim3(kRingThreads), smem, s, a, w32,
                              1.0f / static_cast<float>(a.cols));
}

template <int DT, int W, int TPR, int NV, int R, int D>
cudaError_t ring_backward_launch(const NormGradArgs& a, bool w32, cudaStream_t s) {
    static std::atomic<bool> allowed[kMaxDevices];
    constexpr size_t smem = static_cast<size_t>(D) * R * 2 * NV * kRingThreads * 16;
    const cudaError_t e = allow_smem(ring_backward_kernel<DT, W, TPR, NV, R, D>, smem, allowed);
    if (e != cudaSuccess) return e;
    return launch_kernel_smem(ring_backward_kernel<DT, W, TPR, NV, R, D>, dim3(kSMs), dim3(kRingThreads), smem, s, a, w32,
                              1.0f / static_cast<float>(a.cols));
}

// `vecs` vectors of four words a row, at most kRingVecs.
template <int DT, int W> cudaError_t ring_forward_any(const NormArgs& a, bool w32, size_t vecs, cudaStream_t s) {
    if (vecs <= 32) return ring_forward_launch<DT, W, 32, 1, 4, 6>(a, w32, s);
    if (vecs <= 64) return ring_forward_launch<DT, W, 64, 1, 4, 6>(a, w32, s);
    if (vecs <= 128) return ring_forward_launch<DT, W, 128, 1, 4, 6>(a, w32, s);
    if (vecs <= 256) return ring_forward_launch<DT, W, 256, 1, 4, 6>(a, w32, s);
    if (vecs <= 512) return ring_forward_launch<DT, W, 512, 1, 4, 6>(a, w32, s);
    if (vecs <= 1024) return ring_forward_launch<DT, W, 512, 2, 2, 6>(a, w32, s);
    return ring_forward_launch<DT, W, 512, 4, 1, 6>(a, w32, s);
}

template <int DT, int W> cudaError_t ring_backward_any(const NormGradArgs& a, bool w32, size_t vecs, cudaStream_t s) {
    if (vecs <= 32) return ring_backward_launch<DT, W, 32, 1, 4, 3>(a, w32, s);
    if (vecs <= 64) return ring_backward_launch<DT, W, 64, 1, 4, 3>(a, w32, s);
    if (vecs <= 128) return ring_backward_launch<DT, W, 128, 1, 4, 3>(a, w32, s);
    if (vecs <= 256) return ring_backward_launch<DT, W, 256, 1, 4, 3>(a, w32, s);
    if (vecs <= 512) return ring_backward_launch<DT, W, 512, 1, 4, 3>(a, w32, s);
    if (vecs <= 1024) return ring_backward_launch<DT, W, 512, 2, 2, 3>(a, w32, s);
    return ring_backward_launch<DT, W, 512, 4, 1, 3>(a, w32, s);
}

}  // namespace norm
}  // namespace sar
