// orthogonalize.cu -- Newton-Schulz iteration of a batch of matrices:
//   X = g / (|g| + eps);  steps times: A = X X^T, X = (a I + b A + c A A) X.
//
// All but a little of the work is in the three products of a step.  They run on
// the tensor cores, whose inputs have 11 bits, at binary32's precision: every
// value is held as the sum of two fp16 numbers (hi = fp16(v), lo = fp16(v - hi):
// off by 2^-24 of v at most), and a product is hi hi + hi lo + lo hi.  Less will
// not do: the steps multiply small singular values by 3.4 each, the errors in
// their directions with them, so that one fp16 product a step would leave 0.2%
// (1024 columns) to 0.9% (64) of error.  Every matrix is held times a power of
// two of its own, found from a bound of its iterates' singular values, so that
// fp16's range holds it with 2^-39 of the bound for the smallest difference.
//
// The tensor cores' accumulators lose their last bits to truncation, always
// towards zero.  A sum of squares (the diagonal of A) over thousands of columns
// would be off by 2^-15, so the accumulators are taken out every 64 columns and
// added in registers, rounded to nearest, while the next 64 are multiplied.
//
// Matrices between the kernels lie in blocks of 128 rows x 64 columns, 16 KiB of
// hi and 16 KiB of lo, each as the tensor cores want it in shared memory: a tile
// is fetched by bulk copies without a tensor map, and the same block serves as
// an operand along its rows (X X^T) and along its columns (.. X).  A and the
// polynomial are symmetric: their blocks below the diagonal are neither computed
// nor written; where they are wanted, the block across the diagonal is taken
// along its columns.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "sar_device.cuh"
#include "sar_internal.h"
#include "tensor_core.cuh"

namespace sar {
namespace {

constexpr int kSMs = 152;
constexpr int kNormThreads = 256;
constexpr size_t kMaxParts = 256;
constexpr size_t kHalfBlock = 16384, kBlock = 2 * kHalfBlock;

struct Sizes {
    size_t m, n;                       // the smaller side, and the larger
    size_t rb, cb;                     // X: blocks of 128 rows, of 64 columns
    size_t x_blocks, a_blocks;         // of X; of A (rb * 2 rb)
};

Sizes sizes_of(size_t rows, size_t cols) {
    Sizes s;
    s.m = std::min(rows, cols), s.n = std::max(rows, cols);
    s.rb = (s.m + 127) / 128, s.cb = (s.n + 63) / 64;
    s.x_blocks = s.rb * s.cb, s.a_blocks = s.rb * 2 * s.rb;
    return s;
}

size_t norm_parts(size_t rows, size_t cols) { return std::min(kMaxParts, std::max<size_t>(1, rows * cols / 8192)); }

// What the products of one step of one matrix multiply by: powers of two (times
// a coefficient) between the scales of X, A and the polynomial.
struct StepFactors {
    float gram, square, linear, diagonal, apply, first, last, second;
};
constexpr size_t kMaxSteps = 64;

// The workspace: a word that says whether a wait ran out, the sums of squares,
// the steps' factors, and two X, A and the polynomial of A.
struct Space {
    int* failed;
    float* sums;
    StepFactors* factors;
    unsigned char *x, *y, *a, *p;
};

constexpr size_t kHead = 16;

size_t sums_bytes(size_t batch) { return (batch * kMaxParts * 3 * sizeof(float) + 15) / 16 * 16; }

Space space_of(void* workspace, size_t batch, const Sizes& s) {
    unsigned char* w = static_cast<unsigned char*>(workspace);
    Space p;
    p.failed = reinterpret_cast<int*>(w);
    p.sums = reinterpret_cast<float*>(w + kHead);
    p.factors = reinterpret_cast<StepFactors*>(w + kHead + sums_bytes(batch));
    p.x = reinterpret_cast<unsigned char*>(p.factors + batch * kMaxSteps);
    p.y = p.x + batch * s.x_blocks * kBlock;
    p.a = p.y + batch * s.x_blocks * kBlock;
    p.p = p.a + batch * s.a_blocks * kBlock;
    return p;
}

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

// parts x 3 sums for each matrix.
template <int DT>
__global__ void __launch_bounds__(kNormThreads) squares_kernel(OrthogonalizeArgs a, float* sums, int* failed) {
    pdl_wait();
    __shared__ float shared[kNormThreads / 32];
    const size_t z = blockIdx.y, threads = static_cast<size_t>(gridDim.x) * kNormThreads, base = z * a.gstride;
    const size_t down = threads / a.cols, across = threads % a.cols;       // a thread's next element
    const size_t first = static_cast<size_t>(blockIdx.x) * kNormThreads + threadIdx.x;
    size_t r = first / a.cols, c = first % a.cols;
    Squares q;
    while (r < a.rows) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = r < a.rows ? load_elem<DT>(a.g, base + r * a.ldg + c) : 0.0f;
            r += down, c += across;
            if (c >= a.cols) c -= a.cols, ++r;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) q.add(v[i]);
    }
    const float big = block_sum(q.big, shared), mid = block_sum(q.mid, shared), small = block_sum(q.small, shared);
    if (threadIdx.x == 0) {
        float* out = sums + (z * gridDim.x + blockIdx.x) * 3;
        out[0] = big, out[1] = mid, out[2] = small;
        if (z == 0 && blockIdx.x == 0) *failed = 0;
    }
}

// The largest power of two that fp16 holds values up to `most` times, with 9% to
// spare for the bound's and the values' roundings.
__device__ __forceinline__ int scale_below(float most) { return most < 1e-38f ? 140 : ilogbf(60000.0f / most); }

// 2^scale / (norm + eps) = f * first * second, the latter two powers of two: no
// step leaves binary32's range where the product does not.  `top`: a bound of
// the singular values of g / (norm + eps), and `scale` what X is held times.
struct Beginning {
    float f, first, second, top;
    int scale;
    __device__ __forceinline__ float of(float x) const { return x * first * f * second; }
};

// All threads of a block of kNormThreads, parts <= kNormThreads.
__device__ Beginning beginning(const float* sums, int parts, float eps) {
    __shared__ double shared[kNormThreads / 32];
    const int t = threadIdx.x;
    double s = 0.0;
    if (t < parts)
        s = static_cast<double>(sums[3 * t]) * 0x1p180 + sums[3 * t + 1] + static_cast<double>(sums[3 * t + 2]) * 0x1p-160;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    if ((t & 31) == 0) shared[t >> 5] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < kNormThreads / 32; ++w) s += shared[w];
    const double norm = sqrt(s), inv = 1.0 / (norm + static_cast<double>(eps));
    if (!(inv > 0.0) || isinf(inv) || isinf(norm)) return {static_cast<float>(inv), 1.0f, 1.0f, 1.0f, 0};
    const float top = static_cast<float>(norm * inv);
    Beginning b;
    b.top = top > 0.0f && top < 1.0f ? top : 1.0f;
    b.scale = scale_below(b.top);
    int e;
    b.f = static_cast<float>(frexp(inv, &e));
    e += b.scale;
    b.first = ldexpf(1.0f, e / 2), b.second = ldexpf(1.0f, e - e / 2);
    return b;
}

// The factors of a matrix's steps.  |p(s)| <= s (|a| + |b| s^2 + |c| s^4), and
// never above `grown`.
__device__ void step_factors(const OrthogonalizeArgs& a, const Beginning& begin, StepFactors* to) {
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
        f.last = a.scale, f.first = ldexpf(1.0f, (-poly - x) / 2), f.second = ldexpf(1.0f, -poly - x - (-poly - x) / 2);
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

// A block of X from g: a block of the grid each.  Where g has more rows than
// columns, X is its transpose.
template <int DT>
__global__ void __launch_bounds__(kNormThreads) begin_kernel(OrthogonalizeArgs a, const float* sums, int parts,
                                                             StepFactors* factors, unsigned cb, unsigned char* x) {
    pdl_wait();
    __shared__ float tile[128][65];
    const size_t z = blockIdx.y, r0 = static_cast<size_t>(blockIdx.x / cb) * 128, c0 = static_cast<size_t>(blockIdx.x % cb) * 64;
    const Beginning f = beginning(sums + z * parts * 3, parts, a.eps);
    const int t = threadIdx.x;
    if (blockIdx.x == 0 && t == 0) step_factors(a, f, factors + z * kMaxSteps);
    const size_t base = z * a.gstride;
    if (a.rows <= a.cols) {
#pragma unroll 8
        for (int i = 0; i < 32; ++i) {
            const int r = t / 64 + 4 * i, c = t % 64;
            tile[r][c] = r0 + r < a.rows && c0 + c < a.cols ? f.of(load_elem<DT>(a.g, base + (r0 + r) * a.ldg + c0 + c)) : 0.0f;
        }
    } else {
#pragma unroll 8
        for (int i = 0; i < 32; ++i) {
            const int r = t % 128, c = t / 128 + 2 * i;
            tile[r][c] = r0 + r < a.cols && c0 + c < a.rows ? f.of(load_elem<DT>(a.g, base + (c0 + c) * a.ldg + r0 + r)) : 0.0f;
        }
    }
    __syncthreads();
    unsigned char* block = x + (z * gridDim.x + blockIdx.x) * kBlock;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = t + kNormThreads * i, r = at / 8, p = at % 8;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = tile[r][8 * p + j];
        uint4 hi, lo;
        split8(v, hi, lo);
        uint4* to = reinterpret_cast<uint4*>(block + r * 128 + ((p ^ (r & 7)) << 4));
        to[0] = hi;
        to[kHalfBlock / 16] = lo;
    }
}

// ---------------------------------------------------------------------------
// The products.
// ---------------------------------------------------------------------------
enum Mode {
    kGram,    // A = X X^T
    kPoly,    // P = a I + b A + c A A
    kApply,   // X = P X
    kLast     // out = scale P X
};

struct ProductArgs {
    const unsigned char* p;      // left operand, rows of k
    const unsigned char* q;      // right operand: rows of k (kGram, kPoly), or k rows (kApply, kLast)
    unsigned char* to;           // not kLast
    int* failed;
    unsigned tiles, per_matrix;  // of all matrices, of one
    int m, n;                    // rows and columns of the product
    int rb, cb;                  // blocks of 128 rows of P, blocks of 64 columns of X
    int kb;                      // blocks of 64 along k
    size_t p_stride, q_stride, to_stride;      // bytes from one matrix to the next
    const StepFactors* factors;  // of this step, kMaxSteps from one matrix to the next
    // kLast
    void* out;
    size_t ldo, ostride;
    bool transposed;
};

// A tile is 128 rows x NT columns.  Warp 0 fetches, warp 1 multiplies (2 and 3
// only make up the group of four whose registers are given away), eight warps
// take the accumulators out: 32 rows and half of the columns each.
constexpr int kTakers = 8, kThreads = 128 + 32 * kTakers;
// Registers of a thread: at the launch, then of the first four warps and of the
// takers, which hold up to 128 sums.  The shares are below what was launched.
constexpr int kLaunchRegisters = 168, kFewRegisters = 40, kManyRegisters = 224;
static_assert(128 * kFewRegisters + 32 * kTakers * kManyRegisters <= kThreads * kLaunchRegisters, "registers");
constexpr int kStaging = 4096;         // of each taker: 32 rows x 32 columns, hi and lo, or binary32

template <int NT> constexpr int kStageBytes = static_cast<int>(kBlock) + NT * 256;
template <int NT> constexpr int kStages = NT == 256 ? 2 : 3;
template <int NT> constexpr size_t kSmem = 1024 + size_t(kStages<NT>) * kStageBytes<NT> + kTakers * kStaging;

struct Place {
    size_t z;
    int row, col;                      // first block of rows; first column / NT
};

// The tiles of a symmetric product: those that reach the diagonal or lie above.
template <int NT, bool SYMMETRIC> __device__ __forceinline__ Place place_of(const ProductArgs& a, unsigned tile) {
    Place p;
    p.z = tile / a.per_matrix;
    int left = static_cast<int>(tile % a.per_matrix);
    constexpr int per = NT / 128;
    if (SYMMETRIC) {
        const int across = (a.rb + per - 1) / per;
        p.row = 0;
        while (left >= across - p.row / per) left -= across - p.row / per, ++p.row;
        p.col = p.row / per + left;
    } else {
        const int across = (a.n + NT - 1) / NT;
        p.row = left / across;
        p.col = left % across;
    }
    return p;
}

// Whether the operands of a block of k are taken along their columns: X on the
// right of the polynomial, and what lies below the diagonal of a symmetric
// matrix.  (The NT / 128 rows of blocks on the right of A A are on one side of the
// diagonal, or on it, which is stored whole.)
struct Turned {
    bool left, right;
};
template <int MODE, int NT> __device__ __forceinline__ Turned turned_of(const ProductArgs& a, const Place& at, int k) {
    if (MODE == kGram) return {false, false};
    if (MODE == kPoly) return {k / 2 < at.row, k / 2 < min((at.col + 1) * (NT / 128), a.rb) - 1};
    return {k / 2 < at.row, true};
}

// A taker's 32 x 32 values in its staging, each half 32 rows of 64 bytes whose
// 16-byte pieces are exchanged so that neither its rows nor its lines collide.
__device__ __forceinline__ int staged(int row, int piece) { return row * 64 + ((piece ^ ((row >> 1) & 3)) << 4); }

// From the staging to rows row0 .. of a block; half: its first or second 32 columns.
__device__ __forceinline__ void store_staged(const unsigned char* staging, unsigned char* block, int row0, int half, int lane) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + lane / 4, p = lane % 4, row = row0 + r;
        unsigned char* to = block + row * 128 + (((half * 4 + p) ^ (row & 7)) << 4);
        *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(staging + staged(r, p));
        *reinterpret_cast<uint4*>(to + kHalfBlock) = *reinterpret_cast<const uint4*>(staging + 2048 + staged(r, p));
    }
    __syncwarp();
}

__device__ __forceinline__ void load_staged(unsigned char* staging, const unsigned char* block, int row0, int half, int lane) {
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = row0 + i * 8 + lane / 4, p = lane % 4;
        const unsigned char* from = block + row * 128 + (((half * 4 + p) ^ (row & 7)) << 4);
        v[2 * i] = *reinterpret_cast<const uint4*>(from);
        v[2 * i + 1] = *reinterpret_cast<const uint4*>(from + kHalfBlock);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + lane / 4, p = lane % 4;
        *reinterpret_cast<uint4*>(staging + staged(r, p)) = v[2 * i];
        *reinterpret_cast<uint4*>(staging + 2048 + staged(r, p)) = v[2 * i + 1];
    }
    __syncwarp();
}

// What a taker does with 32 of its row's sums, columns col0 .. of row `row`
// (both multiples of 32 but for the lane in the row).
template <int MODE, int DT>
__device__ __forceinline__ void finish(const ProductArgs& a, const Place& at, const StepFactors& f, float (&v)[32], int row0, int col0,
                                       unsigned char* staging, int lane, bool failed) {
    if (MODE == kLast) {
        if (col0 >= a.n) return;
        const int rows = a.m - row0, cols = a.n - col0;
        const size_t base = at.z * a.ostride;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = failed ? __uint_as_float(0x7FFFFFFFu) : __fmul_rn(__fmul_rn(__fmul_rn(v[j], f.first), f.last), f.second);
        if (a.transposed) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (lane < rows && j < cols)
                    store_elem<DT>(a.out, base + static_cast<size_t>(col0 + j) * a.ldo + static_cast<size_t>(row0 + lane), v[j]);
            return;
        }
        float* mine = reinterpret_cast<float*>(staging);
#pragma unroll
        for (int p = 0; p < 8; ++p)
            *reinterpret_cast<float4*>(mine + lane * 32 + ((p ^ (lane & 7)) << 2)) =
                make_float4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
        __syncwarp();
#pragma unroll 8
        for (int r = 0; r < 32; ++r)
            if (r < rows && lane < cols)
                store_elem<DT>(a.out, base + static_cast<size_t>(row0 + r) * a.ldo + static_cast<size_t>(col0 + lane),
                               mine[r * 32 + ((((lane >> 2) ^ (r & 7)) << 2) | (lane & 3))]);
        __syncwarp();
        return;
    }
    constexpr bool square = MODE == kGram || MODE == kPoly;
    const int row_block = row0 / 128, col_block = col0 / 64, half = col0 / 32 % 2, across = square ? 2 * a.rb : a.cb;
    if (col_block >= across) return;
    if (square && col0 / 128 < row_block) return;                 // below the diagonal
    const size_t block = static_cast<size_t>(row_block) * across + col_block;
    unsigned char* to = a.to + at.z * a.to_stride;
    if (MODE == kPoly) {
        load_staged(staging, a.p + at.z * a.p_stride + block * kBlock, row0 % 128, half, lane);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint4 hi = *reinterpret_cast<const uint4*>(staging + staged(lane, p));
            const uint4 lo = *reinterpret_cast<const uint4*>(staging + 2048 + staged(lane, p));
            const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x[2], y[2];
                widen_word<SAR_FP16>(h[j], x);
                widen_word<SAR_FP16>(l[j], y);
                float* s = v + 8 * p + 2 * j;
                s[0] = __fmaf_rn(f.square, s[0], __fmul_rn(f.linear, __fadd_rn(x[0], y[0])));
                s[1] = __fmaf_rn(f.square, s[1], __fmul_rn(f.linear, __fadd_rn(x[1], y[1])));
            }
        }
        if (row0 == col0 && row0 + lane < a.m) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (j == lane) v[j] = __fadd_rn(v[j], f.diagonal);
        }
        __syncwarp();
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __fmul_rn(MODE == kGram ? f.gram : f.apply, v[j]);
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        uint4 hi, lo;
        split8(v + 8 * p, hi, lo);
        *reinterpret_cast<uint4*>(staging + staged(lane, p)) = hi;
        *reinterpret_cast<uint4*>(staging + 2048 + staged(lane, p)) = lo;
    }
    store_staged(staging, to + block * kBlock, row0 % 128, half, lane);
}

template <int MODE, int NT, int DT> __global__ void __launch_bounds__(kThreads, 1) product_kernel(ProductArgs a) {
    constexpr bool square = MODE == kGram || MODE == kPoly;       // B's rows run along k
    constexpr int stages = kStages<NT>;
    extern __shared__ unsigned char dynamic[];
    __shared__ uint64_t bars[2 * stages + 5];
    __shared__ uint32_t tmem;
    __shared__ int aborted;
    unsigned char* smem = dynamic + (1024 - tc::shared_address(dynamic) % 1024) % 1024;
    unsigned char* staging = smem + stages * kStageBytes<NT>;
    const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
    const uint32_t bar0 = tc::shared_address(bars);
    const auto full = [&](int s) { return bar0 + 8u * static_cast<uint32_t>(s); };
    const auto empty = [&](int s) { return bar0 + 8u * static_cast<uint32_t>(stages + s); };
    const auto taken = [&](int b) { return bar0 + 8u * static_cast<uint32_t>(2 * stages + b); };
    const auto made = [&](int b) { return bar0 + 8u * static_cast<uint32_t>(2 * stages + 2 + b); };
    const uint32_t drained = bar0 + 8u * (2 * stages + 4);
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) tc::barrier_init(full(s), 1), tc::barrier_init(empty(s), 1);
        for (int b = 0; b < 2; ++b) tc::barrier_init(made(b), 1), tc::barrier_init(taken(b), kTakers);
        tc::barrier_init(drained, 1);
        aborted = 0;
        tc::barrier_init_fence();
    }
    if (warp == 1) tc::tmem_alloc<512>(&tmem);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    pdl_wait();
    const uint32_t acc0 = tmem;
    volatile int* abort_word = &aborted;

    if (warp < 4) tc::fewer_registers<kFewRegisters>();
    if (warp == 0) {
        if (lane == 0) {
            tc::fence_async();
            uint32_t issued = 0;
            bool ok = true;
            for (unsigned tile = blockIdx.x; tile < a.tiles && ok; tile += gridDim.x) {
                const Place at = place_of<NT, square>(a, tile);
                const unsigned char *left = a.p + at.z * a.p_stride, *right = a.q + at.z * a.q_stride;
                const int across = MODE == kGram ? a.cb : 2 * a.rb;
                const int have = square ? min(NT / 128, a.rb - at.col * (NT / 128)) : min(NT / 64, a.cb - at.col * (NT / 64));
                for (int k = 0; k < a.kb && ok; ++k) {
                    const int s = static_cast<int>(issued % stages);
                    ok = issued < static_cast<uint32_t>(stages) || tc::barrier_wait(empty(s), (issued / stages - 1) & 1, abort_word);
                    if (!ok) break;
                    const uint32_t to = tc::shared_address(smem + s * kStageBytes<NT>), b_hi = to + kBlock, b_lo = b_hi + NT * 128;
                    const Turned turned = turned_of<MODE, NT>(a, at, k);
                    // 64 rows (of k) of `count` blocks in a row, hi and lo
                    const auto along_columns = [&](uint32_t hi, uint32_t lo, const unsigned char* from, int across_from, int first, int count) {
                        const unsigned char* src = from + (static_cast<size_t>(k / 2) * across_from + first) * kBlock + (k % 2) * (kHalfBlock / 2);
                        for (int j = 0; j < count; ++j) {
                            tc::bulk_load(hi + j * (kHalfBlock / 2), src + j * kBlock, kHalfBlock / 2, full(s));
                            tc::bulk_load(lo + j * (kHalfBlock / 2), src + j * kBlock + kHalfBlock, kHalfBlock / 2, full(s));
                        }
                    };
                    tc::barrier_expect(full(s), static_cast<uint32_t>(kBlock) + static_cast<uint32_t>(square ? kBlock : kHalfBlock) * have);
                    if (turned.left)
                        along_columns(to, to + kHalfBlock, left, across, 2 * at.row, 2);
                    else
                        tc::bulk_load(to, left + (static_cast<size_t>(at.row) * across + k) * kBlock, kBlock, full(s));
                    if (!square) {
                        along_columns(b_hi, b_lo, right, a.cb, at.col * (NT / 64), have);
                    } else if (turned.right) {
                        along_columns(b_hi, b_lo, right, across, at.col * (NT / 64), 2 * have);
                    } else {
                        for (int j = 0; j < have; ++j) {
                            const unsigned char* from = right + (static_cast<size_t>(at.col * (NT / 128) + j) * across + k) * kBlock;
                            tc::bulk_load(b_hi + j * kHalfBlock, from, kHalfBlock, full(s));
                            tc::bulk_load(b_lo + j * kHalfBlock, from + kHalfBlock, kHalfBlock, full(s));
                        }
                    }
                    ++issued;
                }
            }
            // Nothing is in flight when the block ends: the last copies have been
            // multiplied, or at least have arrived.
            for (uint32_t i = issued > static_cast<uint32_t>(stages) ? issued - stages : 0; i < issued; ++i) {
                const int s = static_cast<int>(i % stages);
                if (ok) ok = tc::barrier_wait(empty(s), (i / stages) & 1, abort_word);
                if (!ok) tc::barrier_wait(full(s), (i / stages) & 1, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t used = 0;
            bool ok = true;
            for (unsigned tile = blockIdx.x; tile < a.tiles && ok; tile += gridDim.x) {
                const Place at = place_of<NT, square>(a, tile);
                for (int k = 0; k < a.kb && ok; ++k) {
                    const uint32_t b = used & 1;
                    ok = used < 2 || tc::barrier_wait(taken(b), (used / 2 - 1) & 1, abort_word);
                    if (!ok) break;
                    tc::fence_after();
                    const int s = static_cast<int>(used % stages);
                    ok = tc::barrier_wait(full(s), (used / stages) & 1, abort_word);
                    if (!ok) break;
                    tc::fence_after();
                    const uint32_t from = tc::shared_address(smem + s * kStageBytes<NT>), acc = acc0 + b * NT;
                    const uint32_t a_hi = from, a_lo = from + kHalfBlock, b_hi = from + kBlock, b_lo = b_hi + NT * 128;
                    const Turned turned = turned_of<MODE, NT>(a, at, k);
                    const uint32_t instruction = tc::instruction_f16(128, NT, turned.left, turned.right);
                    const uint32_t a_step = turned.left ? 2048 : 32, b_step = turned.right ? 2048 : 32;          // 16 along k
                    const auto operand_a = [&](uint32_t from_a) { return tc::operand(from_a, turned.left ? kHalfBlock / 2 : 0, 1024); };
                    const auto operand_b = [&](uint32_t from_b) { return tc::operand(from_b, turned.right ? kHalfBlock / 2 : 0, 1024); };
                    // hi lo and lo hi first, while the sums are small and their
                    // truncation with them; then hi hi.
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        tc::mma_f16(acc, operand_a(a_hi + a_step * i), operand_b(b_lo + b_step * i), instruction, i != 0);
                        tc::mma_f16(acc, operand_a(a_lo + a_step * i), operand_b(b_hi + b_step * i), instruction, true);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tc::mma_f16(acc, operand_a(a_hi + a_step * i), operand_b(b_hi + b_step * i), instruction, true);
                    tc::mma_commit(empty(s));
                    tc::mma_commit(made(b));
                    ++used;
                }
            }
            if (!ok) {                                                         // products in flight
                tc::mma_commit(drained);
                tc::barrier_wait(drained, 0, nullptr);
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        tc::more_registers<kManyRegisters>();
        const int taker = warp - 4, quarter = warp & 3, half = taker / 4;
        unsigned char* mine = staging + taker * kStaging;
        constexpr int groups = NT / 64;                                       // of 32 columns, for each taker
        uint32_t chunk = 0;
        bool ok = true;
        for (unsigned tile = blockIdx.x; tile < a.tiles && ok; tile += gridDim.x) {
            const Place at = place_of<NT, square>(a, tile);
            float sums[groups][32];
#pragma unroll
            for (int g = 0; g < groups; ++g)
#pragma unroll
                for (int j = 0; j < 32; ++j) sums[g][j] = 0.0f;
            for (int i = 0; i < a.kb && ok; ++i, ++chunk) {
                const uint32_t b = chunk & 1;
                ok = __all_sync(0xFFFFFFFFu, tc::barrier_wait(made(b), (chunk / 2) & 1, abort_word));
                if (!ok) break;
                tc::fence_after();
                const uint32_t from = acc0 + b * NT + half * (NT / 2) + (static_cast<uint32_t>(quarter) << 21);
#pragma unroll
                for (int g = 0; g < groups; ++g) {
                    float v[32];
                    tc::tmem_load(from + 32 * g, v);
#pragma unroll
                    for (int j = 0; j < 32; ++j) sums[g][j] = __fadd_rn(sums[g][j], v[j]);
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::barrier_arrive(taken(b));
            }
            if (!ok) break;
            const StepFactors f = a.factors[at.z * kMaxSteps];
            const bool failed = MODE == kLast && *static_cast<volatile int*>(a.failed) != 0;
            const int row0 = at.row * 128 + quarter * 32, col0 = at.col * NT + half * (NT / 2);
#pragma unroll
            for (int g = 0; g < groups; ++g) finish<MODE, DT>(a, at, f, sums[g], row0, col0 + 32 * g, mine, lane, failed);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && aborted != 0) *static_cast<volatile int*>(a.failed) = 1;
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_free<512>(acc0);
    }
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------
template <int MODE, int NT, int DT> cudaError_t launch_product(const ProductArgs& a, cudaStream_t s) {
    static std::atomic<bool> allowed[kDevices];
    static std::atomic<int> registers;
    cudaError_t e = allow_smem(product_kernel<MODE, NT, DT>, kSmem<NT>, allowed);
    if (e != cudaSuccess) return e;
    if (registers.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes f;
        if ((e = cudaFuncGetAttributes(&f, product_kernel<MODE, NT, DT>)) != cudaSuccess) return e;
        registers.store(f.numRegs, std::memory_order_relaxed);
    }
    // The takers' registers come out of what the launch has: never wait for more.
    if (registers.load(std::memory_order_relaxed) != kLaunchRegisters) return cudaErrorInvalidConfiguration;
    const unsigned grid = std::min<unsigned>(a.tiles, kSMs);
    return launch_kernel_smem(product_kernel<MODE, NT, DT>, dim3(grid), dim3(kThreads), kSmem<NT>, s, a);
}

template <int MODE, int NT, int DT = SAR_FP32> cudaError_t product(ProductArgs a, size_t batch, cudaStream_t s) {
    const int per = NT / 128, across = (a.rb + per - 1) / per;
    unsigned tiles = 0;
    if (MODE == kGram || MODE == kPoly) {
        for (int r = 0; r < a.rb; ++r) tiles += static_cast<unsigned>(across - r / per);
    } else {
        tiles = static_cast<unsigned>(a.rb) * static_cast<unsigned>((a.n + NT - 1) / NT);
    }
    a.per_matrix = tiles;
    const size_t all = batch * tiles;
    if (all > 0x7FFFFFFF) return cudaErrorInvalidValue;
    a.tiles = static_cast<unsigned>(all);
    return launch_product<MODE, NT, DT>(a, s);
}

template <int DT> cudaError_t launch(const OrthogonalizeArgs& a, cudaStream_t s) {
    const Sizes sz = sizes_of(a.rows, a.cols);
    Space w = space_of(a.workspace, a.batch, sz);
    const unsigned parts = static_cast<unsigned>(norm_parts(a.rows, a.cols)), batch = static_cast<unsigned>(a.batch);
    cudaError_t e = launch_kernel(squares_kernel<DT>, dim3(parts, batch), dim3(kNormThreads), s, a, w.sums, w.failed);
    if (e != cudaSuccess) return e;
    e = launch_kernel(begin_kernel<DT>, dim3(static_cast<unsigned>(sz.x_blocks), batch), dim3(kNormThreads), s, a,
                      static_cast<const float*>(w.sums), static_cast<int>(parts), w.factors, static_cast<unsigned>(sz.cb), w.x);
    if (e != cudaSuccess) return e;
    ProductArgs g = {};
    g.failed = w.failed;
    g.m = static_cast<int>(sz.m), g.n = static_cast<int>(sz.m);
    g.rb = static_cast<int>(sz.rb), g.cb = static_cast<int>(sz.cb);
    const size_t xs = sz.x_blocks * kBlock, as = sz.a_blocks * kBlock;
    for (int k = 0; k < a.steps; ++k) {
        g.factors = w.factors + k;
        ProductArgs gram = g;
        gram.p = gram.q = w.x, gram.to = w.a, gram.p_stride = gram.q_stride = xs, gram.to_stride = as;
        gram.kb = g.cb;
        if ((e = product<kGram, 256>(gram, a.batch, s)) != cudaSuccess) return e;
        ProductArgs poly = g;
        poly.p = poly.q = w.a, poly.to = w.p, poly.p_stride = poly.q_stride = poly.to_stride = as;
        poly.kb = static_cast<int>((sz.m + 63) / 64);
        if ((e = product<kPoly, 256>(poly, a.batch, s)) != cudaSuccess) return e;
        ProductArgs apply = g;
        apply.n = static_cast<int>(sz.n), apply.kb = poly.kb;
        apply.p = w.p, apply.q = w.x, apply.to = w.y, apply.p_stride = as, apply.q_stride = apply.to_stride = xs;
        if (k + 1 < a.steps) {
            e = product<kApply, 256>(apply, a.batch, s);
        } else {
            apply.out = a.out, apply.ldo = a.ldo, apply.ostride = a.ostride, apply.transposed = a.rows > a.cols;
            e = product<kLast, 256, DT>(apply, a.batch, s);
        }
        if (e != cudaSuccess) return e;
        std::swap(w.x, w.y);
    }
    return cudaSuccess;
}

}  // namespace

size_t orthogonalize_workspace_bytes(size_t batch, size_t rows, size_t cols) {
    const Sizes s = sizes_of(rows, cols);
    return kHead + sums_bytes(batch) + batch * kMaxSteps * sizeof(StepFactors) + batch * (2 * s.x_blocks + 2 * s.a_blocks) * kBlock;
}

cudaError_t launch_orthogonalize(sar_dtype dt, const OrthogonalizeArgs& a, cudaStream_t s) {
    switch (dt) {
    case SAR_BF16: return launch<SAR_BF16>(a, s);
    case SAR_FP16: return launch<SAR_FP16>(a, s);
    default: return launch<SAR_FP32>(a, s);
    }
}

}  // namespace sar
