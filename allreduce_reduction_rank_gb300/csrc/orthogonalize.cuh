// orthogonalize.cuh -- what both forms of the Newton-Schulz iteration share: the
// norm, the powers of two that values are held times, and values as two fp16
// numbers.
#pragma once

#include <cmath>

#include "sar_device.cuh"
#include "sar_internal.h"
#include "tensor_core.cuh"

namespace sar {
namespace orthogonal {

constexpr int kNormThreads = 256;
constexpr size_t kHalfBlock = 16384, kBlock = 2 * kHalfBlock;

// What the products of one step of one matrix multiply by: powers of two (times
// a coefficient) between the scales of X, A and the polynomial; after the last step
// three that together make the result, each between it and the product, so that none
// leaves binary32's range where the result does not.
struct StepFactors {
    float gram, square, linear, diagonal, apply, first, second, third;
};
constexpr size_t kMaxSteps = 64;

// ---------------------------------------------------------------------------
// The norm.
// ---------------------------------------------------------------------------

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
    __device__ __forceinline__ void add(const Squares& o) {
        big = __fadd_rn(big, o.big), mid = __fadd_rn(mid, o.mid), small = __fadd_rn(small, o.small);
    }
};

// A sum of many short Squares.  Additions of about one term again and again err to one
// side for as long as the sum keeps its power of two: 2048 squares of one value in a row by
// 3e-5, 32768 by 5e-4.  What an addition loses is kept, and added to the next term.
struct LongSquares {
    Squares sum, lost;
    static __device__ __forceinline__ void add(float& sum, float& lost, float x) {
        const float y = __fadd_rn(x, lost), s = __fadd_rn(sum, y);
        lost = __fsub_rn(y, __fsub_rn(s, sum));
        sum = s;
    }
    __device__ __forceinline__ void add(const Squares& o) {
        add(sum.mid, lost.mid, o.mid);
        if (o.big != 0.0f) add(sum.big, lost.big, o.big);
        if (o.small != 0.0f) add(sum.small, lost.small, o.small);
    }
};

__device__ __forceinline__ float block_sum(float x, float* shared) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kNormThreads / 32; ++w) s = __fadd_rn(s, shared[w]);
    return s;
}

// The largest power of two that fp16 holds values up to `most` times, with 9% to
// spare for the bound's and the values' roundings.  most > 0; the quotient stays finite.
__device__ __forceinline__ int scale_below(float most) {
    return most < 1e-30f ? 100 + ilogbf(60000.0f / (most * 0x1p100f)) : ilogbf(60000.0f / most);
}

// 2^scale / (norm + eps) = f * first * second, the latter two powers of two: no
// step leaves binary32's range where the product does not.  `top`: a bound of
// the singular values of g / (norm + eps), and `scale` what X is held times.
struct Beginning {
    float f, first, second, top;
    int scale;
    __device__ __forceinline__ float of(float x) const { return x * first * f * second; }
};

// From the sums of Squares.  In binary32, the norm as m 2^k: double precision, a
// sixty-fourth of the rate here, took 40 us of a 4096 x 4096 matrix's beginning.
__device__ __forceinline__ Beginning beginning(float big, float mid, float small, float eps) {
    float square = small, k_eps = eps * 0x1p80f;                     // eps / 2^k
    int k = -80;
    if (big != 0.0f)
        square = big + mid * 0x1p-90f * 0x1p-90f, k_eps = eps * 0x1p-90f, k = 90;
    else if (mid != 0.0f)
        square = mid + small * 0x1p-80f * 0x1p-80f, k_eps = eps, k = 0;
    float m = sqrtf(square);
    if (isinf(k_eps)) m = m * 0x1p-80f, k_eps = eps, k = 0;          // eps above 2^48 beside small values only
    const float whole = m + k_eps, inv = __fdiv_rn(1.0f, whole);
    if (!(inv > 0.0f) || isinf(inv)) return {inv, 1.0f, 1.0f, 1.0f, 0};         // NaN, infinity, zeros with eps 0
    const float top = __fdiv_rn(m, whole);
    Beginning b;
    b.top = top > 0.0f && top < 1.0f ? top : 1.0f;
    b.scale = scale_below(b.top);
    int e;
    b.f = frexpf(inv, &e);
    e += b.scale - k;
    b.first = ldexpf(1.0f, e / 2), b.second = ldexpf(1.0f, e - e / 2);
    return b;
}

// The factors of a matrix's steps.  |p(s)| <= s (|a| + |b| s^2 + |c| s^4), and
// never above `grown`.
__device__ __forceinline__ void step_factors(const OrthogonalizeArgs& a, const Beginning& begin, StepFactors* to) {
    float top = begin.top;
    int x = begin.scale;
    for (int k = 0; k < a.steps; ++k) {
        const float square = top * top, most = fabsf(a.a) + square * (fabsf(a.b) + square * fabsf(a.c));
        const float next = fminf(top * most, a.grown);
        const int gram = 2 * x - 16, poly = scale_below(most), after = scale_below(next);
        StepFactors f;
        f.gram = ldexpf(1.0f, gram - 2 * x);
        f.square = ldexpf(a.c, poly - 2 * gram);
        f.linear = ldexpf(a.b, poly - gram);
        f.diagonal = ldexpf(a.a, poly);
        f.apply = ldexpf(1.0f, after - poly - x);
        int e;                                                       // first * second * third = scale 2^(-poly - x)
        const float scale = frexpf(a.scale, &e);
        e -= poly + x;
        f.first = ldexpf(scale, e / 3), f.second = ldexpf(1.0f, e / 3), f.third = ldexpf(1.0f, e - e / 3 * 2);
        to[k] = f;
        top = next, x = after;
    }
}

// ---------------------------------------------------------------------------
// Values as two fp16 numbers.
// ---------------------------------------------------------------------------

// Eight values into 16 bytes of hi and of lo.
__device__ __forceinline__ void split8(const float* v, uint4& hi, uint4& lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 a = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        const float2 w = __half22float2(a);
        const __half2 b = __floats2half2_rn(__fsub_rn(v[2 * i], w.x), __fsub_rn(v[2 * i + 1], w.y));
        h[i] = *reinterpret_cast<const uint32_t*>(&a);
        l[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

}  // namespace orthogonal

// The form for matrices of up to 128 rows (or columns): one launch.
bool orthogonalize_small_fits(size_t rows, size_t cols);
cudaError_t launch_orthogonalize_small(sar_dtype dt, const OrthogonalizeArgs& a, cudaStream_t s);

}  // namespace sar
