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
// would be off by 2^-15, so the accumulators are taken out every 64 columns (every
// 256 for g of 16 bits, see product below) and added in registers, rounded to nearest,
// while the next are multiplied.
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

#include "orthogonalize.cuh"

namespace sar {
namespace {

using namespace orthogonal;

constexpr int kSMs = 152;
constexpr size_t kMaxParts = 512;

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

// Whether the rows of all matrices start on 16-byte boundaries.
template <int DT> __device__ __forceinline__ bool rows_aligned(const OrthogonalizeArgs& a) {
    return ((reinterpret_cast<uintptr_t>(a.g) | a.ldg * Elem<DT>::kSize | a.gstride * Elem<DT>::kSize) & 15) == 0;
}

// The squares of pieces of kVE columns: those at c0, c0 + step, .. of row r and of
// every `down`-th row below, four pieces a short sum, in an order that alignment does
// not change.
template <int DT, bool kVec>
__device__ __forceinline__ void add_squares(LongSquares& q, const OrthogonalizeArgs& a, size_t base, size_t r, size_t c0, size_t down,
                                            size_t step) {
    constexpr int together = kVec ? 8 : 4, ve = Elem<DT>::kVE;
    for (size_t c = c0; c < a.cols; c += step) {
        const int have = static_cast<int>(a.cols - c < static_cast<size_t>(ve) ? a.cols - c : static_cast<size_t>(ve));
        for (size_t i = r; i < a.rows; i += together * down) {
            Acc<DT> x[together];
#pragma unroll
            for (int j = 0; j < together; ++j) {
                const size_t row = i + static_cast<size_t>(j) * down, at = base + row * a.ldg + c;
                if (kVec && have == ve) {
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (row < a.rows) v = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.g) + at * Elem<DT>::kSize);
                    acc_seed<DT>(x[j], v);
                    continue;
                }
#pragma unroll
                for (int e = 0; e < ve; ++e) x[j].v[e] = row < a.rows && e < have ? load_elem<DT>(a.g, at + e) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < together; j += 4) {
                Squares four;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < ve; ++e) four.add(x[j + i].v[e]);
                q.add(four);
            }
        }
    }
}

// parts x 3 sums for each matrix.  A row of a block's threads, a power of two of
// them, goes along a row of the matrix.
template <int DT>
__global__ void __launch_bounds__(kNormThreads) squares_kernel(OrthogonalizeArgs a, float* sums, int* failed, int along) {
    pdl_wait();
    __shared__ float shared[kNormThreads / 32];
    const size_t z = blockIdx.y, base = z * a.gstride;
    const size_t lines = static_cast<size_t>(kNormThreads / along);
    const size_t r = blockIdx.x * lines + threadIdx.x / along, down = gridDim.x * lines, x = threadIdx.x % along;
    constexpr int ve = Elem<DT>::kVE;
    LongSquares q;
    if (rows_aligned<DT>(a))
        add_squares<DT, true>(q, a, base, r, x * ve, down, static_cast<size_t>(along) * ve);
    else
        add_squares<DT, false>(q, a, base, r, x * ve, down, static_cast<size_t>(along) * ve);
    const float big = block_sum(q.sum.big, shared), mid = block_sum(q.sum.mid, shared), small = block_sum(q.sum.small, shared);
    if (threadIdx.x == 0) {
        float* out = sums + (z * gridDim.x + blockIdx.x) * 3;
        out[0] = big, out[1] = mid, out[2] = small;
        if (z == 0 && blockIdx.x == 0) *failed = 0;
    }
}

// All threads of a block of kNormThreads.
__device__ __forceinline__ Beginning beginning_of(const float* sums, int parts, float eps) {
    __shared__ float shared[kNormThreads / 32];
    const int t = threadIdx.x;
    float big = 0.0f, mid = 0.0f, small = 0.0f;
    for (int i = t; i < parts; i += kNormThreads)
        big = __fadd_rn(big, sums[3 * i]), mid = __fadd_rn(mid, sums[3 * i + 1]), small = __fadd_rn(small, sums[3 * i + 2]);
    const float all_big = block_sum(big, shared), all_mid = block_sum(mid, shared), all_small = block_sum(small, shared);
    return beginning(all_big, all_mid, all_small, eps);
}

// A block of X from g: a block of the grid each.  Where g has more rows than
// columns, X is its transpose.
template <int DT>
__global__ void __launch_bounds__(kNormThreads) begin_kernel(OrthogonalizeArgs a, const float* sums, int parts,
                                                             StepFactors* factors, unsigned cb, unsigned char* x) {
    pdl_wait();
    __shared__ float tile[128][65];
    const size_t z = blockIdx.y, r0 = static_cast<size_t>(blockIdx.x / cb) * 128, c0 = static_cast<size_t>(blockIdx.x % cb) * 64;
    const int t = threadIdx.x;
    const auto norm = [&]() {                                                 // after the loads, which do not need it
        const Beginning f = beginning_of(sums + z * parts * 3, parts, a.eps);
        if (blockIdx.x == 0 && t == 0) step_factors(a, f, factors + z * kMaxSteps);
        return f;
    };
    const size_t base = z * a.gstride;
    unsigned char* block = x + (z * gridDim.x + blockIdx.x) * kBlock;
    if (a.rows <= a.cols && a.cols % 8 == 0 && rows_aligned<DT>(a)) {         // pieces of eight columns, as they are
        constexpr int es = Elem<DT>::kSize, ve = Elem<DT>::kVE;
        uint4 w[4][es / 2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < es / 2; ++j) {
                const size_t r = r0 + t / 8 + 32 * i, c = c0 + 8 * (t % 8) + ve * j;
                w[i][j] = make_uint4(0u, 0u, 0u, 0u);
                if (r < a.rows && c < a.cols)
                    w[i][j] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.g) + (base + r * a.ldg + c) * es);
            }
        const Beginning f = norm();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = t / 8 + 32 * i, p = t % 8;
            float v[8];
#pragma unroll
            for (int j = 0; j < es / 2; ++j) {
                Acc<DT> u;
                acc_seed<DT>(u, w[i][j]);
#pragma unroll
                for (int e = 0; e < ve; ++e) v[ve * j + e] = f.of(u.v[e]);
            }
            uint4 hi, lo;
            split8(v, hi, lo);
            uint4* to = reinterpret_cast<uint4*>(block + r * 128 + ((p ^ (r & 7)) << 4));
            to[0] = hi;
            to[kHalfBlock / 16] = lo;
        }
        return;
    }
    float v[32];
    if (a.rows <= a.cols) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const size_t r = r0 + t / 64 + 4 * i, c = c0 + t % 64;
            v[i] = r < a.rows && c < a.cols ? load_elem<DT>(a.g, base + r * a.ldg + c) : 0.0f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const size_t r = r0 + t % 128, c = c0 + t / 128 + 2 * i;
            v[i] = r < a.cols && c < a.rows ? load_elem<DT>(a.g, base + c * a.ldg + r) : 0.0f;
        }
    }
    const Beginning f = norm();
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        if (a.rows <= a.cols)
            tile[t / 64 + 4 * i][t % 64] = f.of(v[i]);
        else
            tile[t % 128][t / 128 + 2 * i] = f.of(v[i]);
    }
    __syncthreads();
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
    int split;                   // blocks of a cluster that share k
    size_t p_stride, q_stride, to_stride;      // bytes from one matrix to the next
    const StepFactors* factors;  // of this step, kMaxSteps from one matrix to the next
    // kLast
    void* out;
    size_t ldo, ostride;
    bool transposed;
};

// A tile is 128 x 128, 128 x 64 where there are few, or 256 x 256 by a pair of blocks,
// of 128 rows each.  Per block of k a SM fetches 64 KiB either way, for twice as many
// products in a pair: one block's tiles of 128 x 256 took 98 KiB for those, and what all
// SMs drew from L2 bound them (4096 x 4096 bf16: 3.37 ms in all, pairs 2.93).
//
// Warp 0 fetches, warp 1 multiplies for both blocks (in the second it says when its
// operands are there), 2 and 3 only make up the group of four whose registers are
// given away; eight warps take the accumulators out: 32 rows and half of the columns
// each.
constexpr int kTakers = 8, kThreads = 128 + 32 * kTakers;
// Registers of a thread: at the launch, then of the first four warps and of the
// takers, which hold up to 128 sums.  The shares are below what was launched.
constexpr int kLaunchRegisters = 168, kFewRegisters = 40, kManyRegisters = 224;
static_assert(128 * kFewRegisters + 32 * kTakers * kManyRegisters <= kThreads * kLaunchRegisters, "registers");
constexpr int kStaging = 4096;         // of each taker: 32 rows x 32 columns, hi and lo, or binary32
constexpr int kStages = 3, kStageBytes = 2 * static_cast<int>(kBlock);        // 128 rows of each operand, 64 along k
constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStageBytes + kTakers * kStaging;
// One block a SM: blocks of a pair or a cluster that waited for another one's tensor memory
// could wait for each other (as in orthogonalize_small.cu).
static_assert(kSmem >= (size_t(192) << 10), "shared memory");

constexpr int kMostSplit = 4;

// How blocks share a tile: one has it for itself (kNarrow: of 64 columns); two have 128
// rows each; those of a cluster have a part of k each, and add.
enum Form { kSingle, kPair, kSplit, kNarrow };
__host__ __device__ constexpr int tile_columns(Form f) { return f == kPair ? 256 : f == kNarrow ? 64 : 128; }
__host__ __device__ constexpr int tile_rows(Form f) { return f == kPair ? 256 : 128; }

struct Place {
    size_t z;
    int row, col;                      // in tiles
};

// The tiles of a symmetric product: those on the diagonal and above.
template <Form FORM, bool SYMMETRIC> __device__ __forceinline__ Place place_of(const ProductArgs& a, unsigned tile) {
    constexpr int wide = tile_columns(FORM), per = tile_rows(FORM) / wide;
    Place p;
    p.z = tile / a.per_matrix;
    int left = static_cast<int>(tile % a.per_matrix);
    const int across = ((SYMMETRIC ? a.rb * 128 : a.n) + wide - 1) / wide;
    if (SYMMETRIC) {
        p.row = 0;
        while (left >= across - per * p.row) left -= across - per * p.row, ++p.row;
        p.col = per * p.row + left;
    } else {
        p.row = left / across;
        p.col = left % across;
    }
    return p;
}

// Whether the operands of a block of k are taken along their columns: X on the
// right of the polynomial, and what lies below the diagonal of a symmetric
// matrix.  Of a pair's two blocks of rows (or columns) both are on one side of the
// diagonal, or on it, where blocks are stored whole.
struct Turned {
    bool left, right;
};
template <int MODE, Form FORM> __device__ __forceinline__ Turned turned_of(const Place& at, int k) {
    constexpr int per = FORM == kPair ? 2 : 1;
    const bool left = k / 2 < per * (at.row + 1) - 1, right = k / 2 < (FORM == kNarrow ? at.col / 2 : per * (at.col + 1) - 1);
    if (MODE == kGram) return {false, false};
    if (MODE == kPoly) return {left, right};
    return {left, true};
}

// Where four columns of a row are among 128 x 128 sums, in floats: exchanged so that
// a column of rows does not collide.
__device__ __forceinline__ int quad_of(int row, int quad) { return row * 128 + ((quad ^ (row & 7)) << 2); }

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

// The same rows of A, on their way while the sums are made; then in the staging.
struct Rows {
    uint4 v[8];
    __device__ __forceinline__ void load(const unsigned char* block, int row0, int half, int lane) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = row0 + i * 8 + lane / 4, p = lane % 4;
            const unsigned char* from = block + row * 128 + (((half * 4 + p) ^ (row & 7)) << 4);
            v[2 * i] = *reinterpret_cast<const uint4*>(from);
            v[2 * i + 1] = *reinterpret_cast<const uint4*>(from + kHalfBlock);
        }
    }
    __device__ __forceinline__ void stage(unsigned char* staging, int lane) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + lane / 4, p = lane % 4;
            *reinterpret_cast<uint4*>(staging + staged(r, p)) = v[2 * i];
            *reinterpret_cast<uint4*>(staging + 2048 + staged(r, p)) = v[2 * i + 1];
        }
        __syncwarp();
    }
};

// Rows row0 .., columns col0 .. of A (32 each), where they are kept.
__device__ __forceinline__ void load_rows(Rows& rows, const ProductArgs& a, const Place& at, int row0, int col0, int lane) {
    const int row_block = row0 / 128, col_block = col0 / 64;
    if (row_block >= a.rb || col_block >= 2 * a.rb || col0 / 128 < row_block) return;
    rows.load(a.p + at.z * a.p_stride + (static_cast<size_t>(row_block) * 2 * a.rb + col_block) * kBlock, row0 % 128, col0 / 32 % 2, lane);
}

// What a taker does with 32 of its row's sums, columns col0 .. of row `row`
// (both multiples of 32 but for the lane in the row).
template <int MODE, int DT>
__device__ __forceinline__ void finish(const ProductArgs& a, const Place& at, const StepFactors& f, float (&v)[32], int row0, int col0,
                                       unsigned char* staging, int lane, bool failed, const Rows& rows) {
    if (MODE == kLast) {
        if (col0 >= a.n) return;
        const int rows = a.m - row0, cols = a.n - col0;
        const size_t base = at.z * a.ostride;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = failed ? __uint_as_float(0x7FFFFFFFu) : __fmul_rn(__fmul_rn(__fmul_rn(v[j], f.first), f.second), f.third);
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
    if (col_block >= across || row_block >= a.rb) return;
    if (square && col0 / 128 < row_block) return;                 // below the diagonal
    const size_t block = static_cast<size_t>(row_block) * across + col_block;
    unsigned char* to = a.to + at.z * a.to_stride;
    if (MODE == kPoly) {
        rows.stage(staging, lane);
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

template <int MODE, Form FORM, int CHUNK, int DT> __global__ void __launch_bounds__(kThreads, 1) product_kernel(ProductArgs a) {
    constexpr bool PAIR = FORM == kPair, SPLIT = FORM == kSplit, NARROW = FORM == kNarrow;
    constexpr bool square = MODE == kGram || MODE == kPoly;       // the right operand is a symmetric matrix's, or X's rows
    constexpr int stages = kStages, blocks = PAIR ? 2 : 1, wide = tile_columns(FORM), depth = NARROW ? 4 : 512 / wide;
    constexpr int right_half = NARROW ? static_cast<int>(kHalfBlock / 2) : static_cast<int>(kHalfBlock);       // hi of the right operand
    extern __shared__ unsigned char dynamic[];
    __shared__ uint64_t bars[3 * stages + 9];
    __shared__ uint32_t tmem;
    __shared__ int aborted;
    unsigned char* smem = dynamic + (1024 - tc::shared_address(dynamic) % 1024) % 1024;
    unsigned char* staging = smem + stages * kStageBytes;
    const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
    const int rank = PAIR ? static_cast<int>(tc::cluster_rank()) : 0;
    const unsigned sharing = SPLIT ? static_cast<unsigned>(a.split) : blocks;
    const unsigned first_tile = blockIdx.x / sharing, tile_step = gridDim.x / sharing;
    const int part = SPLIT ? static_cast<int>(tc::cluster_rank()) : 0;
    const int k_first = SPLIT ? part * a.kb / a.split : 0, k_end = SPLIT ? (part + 1) * a.kb / a.split : a.kb;
    const uint32_t bar0 = tc::shared_address(bars);
    const auto full = [&](int s) { return bar0 + 8u * static_cast<uint32_t>(s); };                       // fetched
    const auto empty = [&](int s) { return bar0 + 8u * static_cast<uint32_t>(stages + s); };             // multiplied
    const auto other = [&](int s) { return bar0 + 8u * static_cast<uint32_t>(2 * stages + s); };         // fetched by the other block
    const auto taken = [&](int b) { return bar0 + 8u * static_cast<uint32_t>(3 * stages + b); };
    const auto made = [&](int b) { return bar0 + 8u * static_cast<uint32_t>(3 * stages + 4 + b); };
    const uint32_t drained = bar0 + 8u * (3 * stages + 8);
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) tc::barrier_init(full(s), 1), tc::barrier_init(empty(s), 1), tc::barrier_init(other(s), 1);
        for (int b = 0; b < 4; ++b) tc::barrier_init(made(b), 1), tc::barrier_init(taken(b), kTakers * blocks);
        tc::barrier_init(drained, 1);
        aborted = 0;
        tc::barrier_init_fence();
    }
    __syncthreads();
    if (PAIR) tc::cluster_sync();                                 // the other block's barriers are there
    if (warp == 1) tc::tmem_alloc<512, PAIR>(&tmem);
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
            for (unsigned tile = first_tile; tile < a.tiles && ok; tile += tile_step) {
                const Place at = place_of<FORM, square>(a, tile);
                const unsigned char *left = a.p + at.z * a.p_stride, *right = a.q + at.z * a.q_stride;
                const int across = MODE == kGram ? a.cb : 2 * a.rb;
                // This block's rows, and its part of the right operand, in blocks of 128.
                const int row = at.row * blocks + rank, col = NARROW ? at.col / 2 : at.col * blocks + rank;
                const int pieces = NARROW ? 1 : max(0, min(2, (square ? 2 * a.rb : a.cb) - 2 * col));  // blocks of 64 of it that there are
                const bool same = square && at.row == (NARROW ? at.col / 2 : at.col);                  // one block for both operands
                const uint32_t bytes =
                    (row < a.rb ? static_cast<uint32_t>(kBlock) : 0u) + (same ? 0u : static_cast<uint32_t>(kHalfBlock) * pieces);
                for (int k = k_first; k < k_end && ok; ++k) {
                    const int s = static_cast<int>(issued % stages);
                    ok = issued < static_cast<uint32_t>(stages) ||
                         tc::barrier_wait<PAIR>(empty(s), (issued / stages - 1) & 1, abort_word);
                    if (!ok) break;
                    const uint32_t to = tc::shared_address(smem + s * kStageBytes), bar = full(s);
                    const Turned turned = turned_of<MODE, FORM>(at, k);
                    // 64 rows (of k) of `count` blocks in a row, hi and lo
                    const auto along_columns = [&](uint32_t hi, int to_lo, const unsigned char* from, int across_from, int first, int count) {
                        const unsigned char* src = from + (static_cast<size_t>(k / 2) * across_from + first) * kBlock + (k % 2) * (kHalfBlock / 2);
                        for (int j = 0; j < count; ++j) {
                            tc::bulk_load(hi + j * (kHalfBlock / 2), src + j * kBlock, kHalfBlock / 2, bar);
                            tc::bulk_load(hi + to_lo + j * (kHalfBlock / 2), src + j * kBlock + kHalfBlock, kHalfBlock / 2, bar);
                        }
                    };
                    tc::barrier_expect(bar, bytes);
                    if (row < a.rb) {
                        if (turned.left)
                            along_columns(to, kHalfBlock, left, across, 2 * row, 2);
                        else
                            tc::bulk_load(to, left + (static_cast<size_t>(row) * across + k) * kBlock, kBlock, bar);
                    }
                    if (same)
                        ;
                    else if (turned.right)
                        along_columns(to + kBlock, right_half, right, square ? across : a.cb, NARROW ? at.col : 2 * col, pieces);
                    else if (NARROW) {
                        const unsigned char* src = right + (static_cast<size_t>(col) * across + k) * kBlock + at.col % 2 * right_half;
                        tc::bulk_load(to + kBlock, src, right_half, bar);
                        tc::bulk_load(to + kBlock + right_half, src + kHalfBlock, right_half, bar);
                    } else if (pieces > 0)
                        tc::bulk_load(to + kBlock, right + (static_cast<size_t>(col) * across + k) * kBlock, kBlock, bar);
                    ++issued;
                }
            }
            // Nothing is in flight when the block ends: the last copies have been
            // multiplied, or at least have arrived.
            for (uint32_t i = issued > static_cast<uint32_t>(stages) ? issued - stages : 0; i < issued; ++i) {
                const int s = static_cast<int>(i % stages);
                if (ok) ok = tc::barrier_wait<PAIR>(empty(s), (i / stages) & 1, abort_word);
                if (!ok) tc::barrier_wait(full(s), (i / stages) & 1, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        if (lane == 0) {
            uint32_t used = 0, chunk = 0;
            bool ok = true;
            for (unsigned tile = first_tile; tile < a.tiles && ok; tile += tile_step) {
                const Place at = place_of<FORM, square>(a, tile);
                for (int k = k_first; k < k_end && ok; ++k, ++used) {
                    const bool begins = (k - k_first) % CHUNK == 0, ends = (k - k_first + 1) % CHUNK == 0 || k + 1 == k_end;
                    const int slot = static_cast<int>(chunk % depth), s = static_cast<int>(used % stages);
                    ok = !begins || chunk < depth || tc::barrier_wait<PAIR>(taken(slot), (chunk / depth - 1) & 1, abort_word);
                    ok = ok && tc::barrier_wait(full(s), (used / stages) & 1, abort_word) &&
                         (!PAIR || tc::barrier_wait<PAIR>(other(s), (used / stages) & 1, abort_word));
                    if (!ok) break;
                    tc::fence_after();
                    const uint32_t acc = acc0 + slot * wide, left = tc::shared_address(smem + s * kStageBytes);
                    const bool same = square && at.row == (NARROW ? at.col / 2 : at.col);
                    const uint32_t right = left + static_cast<uint32_t>(!same ? kBlock : NARROW ? at.col % 2 * right_half : 0);
                    const uint32_t right_lo = right + static_cast<uint32_t>(NARROW && !same ? right_half : kHalfBlock);
                    const Turned turned = turned_of<MODE, FORM>(at, k);
                    const uint32_t instruction = tc::instruction_f16(tile_rows(FORM), wide, turned.left, turned.right);
                    const uint32_t a_step = turned.left ? 2048 : 32, b_step = turned.right ? 2048 : 32;          // 16 along k
                    const auto operand_a = [&](uint32_t from) { return tc::operand(from, turned.left ? kHalfBlock / 2 : 0, 1024); };
                    const auto operand_b = [&](uint32_t from) { return tc::operand(from, turned.right ? kHalfBlock / 2 : 0, 1024); };
                    // hi lo and lo hi first, while the sums are small and their
                    // truncation with them; then hi hi.
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        tc::mma_f16<PAIR>(acc, operand_a(left + a_step * i), operand_b(right_lo + b_step * i), instruction, i != 0 || !begins);
                        tc::mma_f16<PAIR>(acc, operand_a(left + kHalfBlock + a_step * i), operand_b(right + b_step * i), instruction, true);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tc::mma_f16<PAIR>(acc, operand_a(left + a_step * i), operand_b(right + b_step * i), instruction, true);
                    tc::mma_commit<PAIR>(empty(s));
                    if (ends) tc::mma_commit<PAIR>(made(slot)), ++chunk;
                }
            }
            if (!ok) {                                                         // products in flight
                tc::mma_commit<PAIR>(drained);
                tc::barrier_wait(drained, 0, nullptr);
            }
        }
        __syncwarp();
    } else if (PAIR && warp == 1) {
        if (lane == 0) {                                                       // this block's operands are there
            uint32_t seen = 0;
            bool ok = true;
            for (unsigned tile = first_tile; tile < a.tiles && ok; tile += tile_step)
                for (int k = 0; k < a.kb && ok; ++k, ++seen) {
                    const int s = static_cast<int>(seen % stages);
                    ok = tc::barrier_wait(full(s), (seen / stages) & 1, abort_word);
                    if (ok) tc::barrier_arrive_cluster(tc::place_in(other(s), 0));
                }
        }
        __syncwarp();
    } else if (warp >= 4) {
        tc::more_registers<kManyRegisters>();
        const int taker = warp - 4, quarter = warp & 3, half = taker / 4;
        unsigned char* mine = staging + taker * kStaging;
        constexpr int groups = wide / 64, together = groups > 1 ? 2 : 1;      // of 32 columns, for each taker
        const uint32_t taken0 = PAIR ? tc::place_in(taken(0), 0) : taken(0);
        uint32_t chunk = 0;
        bool ok = true;
        // After a wait that ran out, the results are NaN; intermediate ones need not be
        // there, as the last launch reads that it has happened.
        for (unsigned tile = first_tile; tile < a.tiles && (ok || MODE == kLast); tile += tile_step) {
            const Place at = place_of<FORM, square>(a, tile);
            float sums[groups][32];
#pragma unroll
            for (int g = 0; g < groups; ++g)
#pragma unroll
                for (int j = 0; j < 32; ++j) sums[g][j] = 0.0f;
            const int row0 = (at.row * blocks + rank) * 128 + quarter * 32, col0 = at.col * wide + half * (wide / 2);
            // A's rows, which the polynomial adds, come with the sums (a pair's takers
            // have no registers for them: one group after another, at the end).
            Rows rows[PAIR || SPLIT ? 1 : groups];
            if (MODE == kPoly && !PAIR && !SPLIT) {
#pragma unroll
                for (int g = 0; g < groups; ++g) load_rows(rows[g], a, at, row0, col0 + 32 * g, lane);
            }
            for (int i = 0; i < (k_end - k_first + CHUNK - 1) / CHUNK && ok; ++i, ++chunk) {
                const int slot = static_cast<int>(chunk % depth);
                ok = __all_sync(0xFFFFFFFFu, tc::barrier_wait<PAIR>(made(slot), (chunk / depth) & 1, abort_word));
                if (!ok) break;
                tc::fence_after();
                const uint32_t from = acc0 + slot * wide + half * (wide / 2) + (static_cast<uint32_t>(quarter) << 21);
                // Two loads at a time; the accumulators are free once the last have
                // come, before they are added.
#pragma unroll
                for (int g = 0; g < groups; g += together) {
                    uint32_t v[together][32];
#pragma unroll
                    for (int h = 0; h < together; ++h) tc::tmem_load(from + 32 * (g + h), v[h]);
#pragma unroll
                    for (int h = 0; h < together; ++h) tc::tmem_wait(v[h]);
                    if (g + together >= groups) {
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (PAIR)
                                tc::barrier_arrive_cluster(taken0 + 8 * slot);
                            else
                                tc::barrier_arrive(taken0 + 8 * slot);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < together; ++h)
#pragma unroll
                        for (int j = 0; j < 32; ++j) sums[g + h][j] = __fadd_rn(sums[g + h][j], __uint_as_float(v[h][j]));
                }
            }
            if (!ok && lane == 0) *static_cast<volatile int*>(a.failed) = 1;
            if (SPLIT) {                                                      // the parts of k meet below
                float* all = reinterpret_cast<float*>(smem);
#pragma unroll
                for (int g = 0; g < groups; ++g)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<float4*>(all + quad_of(quarter * 32 + lane, half * 16 + g * 8 + j)) =
                            make_float4(sums[g][4 * j], sums[g][4 * j + 1], sums[g][4 * j + 2], sums[g][4 * j + 3]);
                break;
            }
            if (!ok && MODE != kLast) break;
            const StepFactors f = a.factors[at.z * kMaxSteps];
            const bool failed = MODE == kLast && (!ok || *static_cast<volatile int*>(a.failed) != 0);
#pragma unroll
            for (int g = 0; g < groups; ++g) {
                Rows& of = rows[PAIR || SPLIT ? 0 : g];
                if (MODE == kPoly && PAIR) load_rows(of, a, at, row0, col0 + 32 * g, lane);
                finish<MODE, DT>(a, at, f, sums[g], row0, col0 + 32 * g, mine, lane, failed, of);
            }
        }
        if (SPLIT) {
            tc::cluster_sync();
            const Place at = place_of<FORM, square>(a, first_tile);
            const StepFactors f = a.factors[at.z * kMaxSteps];
            const bool failed = MODE == kLast && *static_cast<volatile int*>(a.failed) != 0;
            const uint32_t from = tc::shared_address(smem);
            for (int b = part + taker * a.split; b < 16; b += kTakers * a.split) {       // 16 parts of 32 x 32, in turn over the blocks
                float v[32];
                Rows rows;
                if (MODE == kPoly) load_rows(rows, a, at, at.row * 128 + b / 4 * 32, at.col * 128 + b % 4 * 32, lane);
                float4 q[kMostSplit][8];                                      // all on their way together
#pragma unroll
                for (int i = 0; i < kMostSplit; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t quad = from + 4u * static_cast<uint32_t>(quad_of(b / 4 * 32 + lane, b % 4 * 8 + j));
                        q[i][j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (i < a.split) q[i][j] = tc::load_cluster(tc::place_in(quad, static_cast<uint32_t>(i)));
                    }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float4 s = q[0][j];
#pragma unroll
                    for (int i = 1; i < kMostSplit; ++i)
                        s.x = __fadd_rn(s.x, q[i][j].x), s.y = __fadd_rn(s.y, q[i][j].y), s.z = __fadd_rn(s.z, q[i][j].z),
                        s.w = __fadd_rn(s.w, q[i][j].w);
                    v[4 * j] = s.x, v[4 * j + 1] = s.y, v[4 * j + 2] = s.z, v[4 * j + 3] = s.w;
                }
                finish<MODE, DT>(a, at, f, v, at.row * 128 + b / 4 * 32, at.col * 128 + b % 4 * 32, mine, lane, failed, rows);
            }
        }
    }
    if (SPLIT && warp < 4) tc::cluster_sync();                    // as the takers
    tc::fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && aborted != 0) *static_cast<volatile int*>(a.failed) = 1;
    if (PAIR || SPLIT) tc::cluster_sync();                        // nothing of another block's is in use any more
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_free<512, PAIR>(acc0);
    }
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------
template <int MODE, Form FORM, int CHUNK, int DT> cudaError_t launch_product(const ProductArgs& a, cudaStream_t s) {
    static std::atomic<bool> allowed[kDevices];
    static std::atomic<int> registers;
    const auto kernel = product_kernel<MODE, FORM, CHUNK, DT>;
    cudaError_t e = allow_smem(kernel, kSmem, allowed);
    if (e != cudaSuccess) return e;
    if (registers.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes f;
        if ((e = cudaFuncGetAttributes(&f, kernel)) != cudaSuccess) return e;
        registers.store(f.numRegs, std::memory_order_relaxed);
    }
    // The takers' registers come out of what the launch has: never wait for more.
    if (registers.load(std::memory_order_relaxed) != kLaunchRegisters) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = FORM == kPair ? 2u : static_cast<unsigned>(a.split), attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(FORM == kPair ? 2 * std::min<unsigned>(a.tiles, kSMs / 2)
                       : FORM == kSplit ? a.tiles * static_cast<unsigned>(a.split) : std::min<unsigned>(a.tiles, kSMs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = FORM == kSingle || FORM == kNarrow ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

size_t tiles_of(bool symmetric, Form form, const ProductArgs& a) {
    const size_t tall = static_cast<size_t>(tile_rows(form)), wide = static_cast<size_t>(tile_columns(form));
    const size_t rows = (static_cast<size_t>(a.rb) * 128 + tall - 1) / tall;
    return symmetric ? tall / wide * rows * (rows + 1) / 2 : rows * ((static_cast<size_t>(a.n) + wide - 1) / wide);
}

// Pairs of blocks or single ones, by their rounds over the SMs.  A pair's tile is two
// of one block's for each SM, and those take longer: 128 columns of the right
// operand are not enough for the tensor cores' full rate from shared memory, and more
// comes from L2.  4096 x 4096, the time of a pair's tile and that of two single ones, which
// is as much for each SM: 37 and 47 us for g of 16 bits; 45 and 50 us in binary32, where every
// block of k ends with the accumulators being taken, and a pair's takers answer across two
// SMs.  All steps (us) by this rule, with pairs always, with pairs never: 4096 x 4096 bf16
// 2876, 2880, 3468, fp32 3652, 3603, 3857; 2048 x 2048 bf16 495, 627, 547, fp32 566, 778,
// 591; 16 x 1024 x 1024 bf16 1019, 1127, 1043, fp32 1121, 1428, 1122; 4096 x 11008 bf16
// 6551, 6454, 8132; 8192 x 2048 bf16 1412, 1660, 1521; 3 x 2048 x 2048 fp32 1537, 1696, 1620;
// 12 x 600 x 600 fp32 370, 455, 351.
template <int MODE, int DT> cudaError_t product(ProductArgs a, size_t batch, cudaStream_t s) {
    constexpr bool symmetric = MODE == kGram || MODE == kPoly;
    // Blocks of 64 of k between two takings of the accumulators.  One leaves 2e-6 to 4e-6
    // of error (2-norm, five steps of 3.4445, 500 to 3000 rows; 6e-6 after twelve), 4 of
    // them 6e-6 to 9e-6 (3e-5): a result of 16 bits is rounded by 1e-4 or 1e-3 of itself.
    // With one, 4096 x 4096 bf16 would take 3606 us (2876), 2048 x 2048 566 (495).
    constexpr int chunk = DT == SAR_FP32 ? 1 : 4, type = MODE == kLast ? DT : SAR_FP32;
    constexpr size_t pair_time = 200, single_time = DT == SAR_FP32 ? 110 : 129;
    const size_t pairs = batch * tiles_of(symmetric, kPair, a), singles = batch * tiles_of(symmetric, kSingle, a);
    if (singles > 0x7FFFFFFF) return cudaErrorInvalidValue;
    const bool pair = a.rb > 1 && pair_time * ((pairs + kSMs / 2 - 1) / (kSMs / 2)) <= single_time * ((singles + kSMs - 1) / kSMs);
    a.per_matrix = static_cast<unsigned>(tiles_of(symmetric, pair ? kPair : kSingle, a));
    a.tiles = static_cast<unsigned>(pair ? pairs : singles);
    if (pair) return launch_product<MODE, kPair, chunk, type>(a, s);
    // Few tiles and a long k: the SMs that are left share it, which adds 2 to 3 us to a
    // product and takes half or three quarters off its 0.7 us a block of k.  300 x 4000
    // fp32 371 -> 240 us, 1024 x 1024 292 -> 263; 500 x 500 (8 blocks) would lose, 185 ->
    // 204.
    a.split = 1;
    while (a.kb >= 16 && a.split < kMostSplit && singles * a.split * 2 <= kSMs) a.split *= 2;
    if (a.split > 1) return launch_product<MODE, kSplit, chunk, type>(a, s);
    // Tiles of half the width, as long as each has a SM: 48 KiB a block of k, half of the
    // sums.  500 x 500 fp32 180 -> 154 us, 2 x 1003 x 357 fp16 182 -> 169, 300 x 4000 fp32
    // 221 -> 211.
    const size_t narrow = batch * tiles_of(symmetric, kNarrow, a);
    if (narrow > kSMs) return launch_product<MODE, kSingle, chunk, type>(a, s);
    a.per_matrix = static_cast<unsigned>(tiles_of(symmetric, kNarrow, a)), a.tiles = static_cast<unsigned>(narrow);
    return launch_product<MODE, kNarrow, chunk, type>(a, s);
}

template <int DT> cudaError_t launch(const OrthogonalizeArgs& a, cudaStream_t s) {
    const Sizes sz = sizes_of(a.rows, a.cols);
    Space w = space_of(a.workspace, a.batch, sz);
    const unsigned parts = static_cast<unsigned>(norm_parts(a.rows, a.cols)), batch = static_cast<unsigned>(a.batch);
    int along = 1;                                        // threads to a row: as its 16-byte pieces need
    while (along < kNormThreads && static_cast<size_t>(along) * Elem<DT>::kVE < a.cols) along *= 2;
    cudaError_t e = launch_kernel(squares_kernel<DT>, dim3(parts, batch), dim3(kNormThreads), s, a, w.sums, w.failed, along);
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
        if ((e = product<kGram, DT>(gram, a.batch, s)) != cudaSuccess) return e;
        ProductArgs poly = g;
        poly.p = poly.q = w.a, poly.to = w.p, poly.p_stride = poly.q_stride = poly.to_stride = as;
        poly.kb = static_cast<int>((sz.m + 63) / 64);
        if ((e = product<kPoly, DT>(poly, a.batch, s)) != cudaSuccess) return e;
        ProductArgs apply = g;
        apply.n = static_cast<int>(sz.n), apply.kb = poly.kb;
        apply.p = w.p, apply.q = w.x, apply.to = w.y, apply.p_stride = as, apply.q_stride = apply.to_stride = xs;
        if (k + 1 < a.steps) {
            e = product<kApply, DT>(apply, a.batch, s);
        } else {
            apply.out = a.out, apply.ldo = a.ldo, apply.ostride = a.ostride, apply.transposed = a.rows > a.cols;
            e = product<kLast, DT>(apply, a.batch, s);
        }
        if (e != cudaSuccess) return e;
        std::swap(w.x, w.y);
    }
    return cudaSuccess;
}

}  // namespace

size_t orthogonalize_workspace_bytes(size_t batch, size_t rows, size_t cols) {
    if (orthogonalize_small_fits(rows, cols)) return kHead;           // which lies in shared memory only
    const Sizes s = sizes_of(rows, cols);
    return kHead + sums_bytes(batch) + batch * kMaxSteps * sizeof(StepFactors) + batch * (2 * s.x_blocks + 2 * s.a_blocks) * kBlock;
}

cudaError_t launch_orthogonalize(sar_dtype dt, const OrthogonalizeArgs& a, cudaStream_t s) {
    if (orthogonalize_small_fits(a.rows, a.cols)) return launch_orthogonalize_small(dt, a, s);
    switch (dt) {
    case SAR_BF16: return launch<SAR_BF16>(a, s);
    case SAR_FP16: return launch<SAR_FP16>(a, s);
    default: return launch<SAR_FP32>(a, s);
    }
}

}  // namespace sar
