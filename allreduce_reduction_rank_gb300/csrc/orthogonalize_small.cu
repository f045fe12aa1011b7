// orthogonalize_small.cu -- the Newton-Schulz iteration of matrices with up to 128
// rows (X and its transpose exchanged where g has more rows than columns) and 4096
// columns, in one launch.
//
// There the launches of the general form, three a step, are the time: 120 us for 8
// matrices of 128 x 128, 297 for one of 8 x 3648, whose X X^T is one tile.  Here a
// cluster of blocks takes a matrix, each up to 256 of its columns, and keeps them in
// shared memory for all steps.  A step is
//   X X^T of each block's columns; the blocks' sums added, a share of the rows by each
//   block, and given to all of them (the only exchange);
//   the polynomial of A, by every block for itself; its product with the own columns.
// The same arithmetic as in orthogonalize.cu: two fp16 numbers for a value, sums of 64
// products in the tensor cores, those added in binary32.
//
// Taken whatever the batch; this form and the general one in binary32 (us): 8 x 128 x 128
// 47, 90; 1000 x 64 x 64 216, 375; 128 x 1024 93, 129; 64 x 128 x 1024 199, 212; 8 x 3648
// 115, 164; 128 x 4096 126, 176.  Clusters of 16 are the exception, of which six or so find
// their SMs at once: 9 x 128 x 4096 241, 211; 64 x 128 x 4096 1237, 560; 64 x 8 x 3648
// 1094, 390.
#include <algorithm>
#include <atomic>

#include "orthogonalize.cuh"

namespace sar {
namespace {

using namespace orthogonal;

constexpr int kThreads = 256;
constexpr int kColumns = 256, kMostBlocks = 16;
constexpr int kMostSteps = 64;
// Shared memory that a cluster's block asks for at least, whatever its columns need (160
// KiB or more): with it in a SM's 228 KiB no other kernel that multiplies there finds room.
// A block takes all of its SM's tensor memory before it waits for its cluster; were two
// clusters' blocks to share SMs, one could wait for columns of the other and the other for
// its.  224 KiB, which leave less of L1, cost up to 3% of matrices of 17 to 64 rows.
constexpr size_t kAlone = size_t(192) << 10;

// A power of two, so that a cluster's rows and exchanges split evenly: 2100 columns take 16
// blocks, of which 11 have some.
int blocks_of(size_t n) {
    int blocks = 1;
    while (static_cast<size_t>(blocks) * kColumns < n) blocks *= 2;
    return blocks;
}

__device__ __forceinline__ void store_cluster(uint32_t at, const uint4& v) {
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Piece p (8 columns) of row r in a block of 128 rows x 64 columns.
__device__ __forceinline__ int piece_at(int r, int p) { return r * 128 + ((p ^ (r & 7)) << 4); }
// Four columns of row r in a matrix of 128 binary32 columns.
__device__ __forceinline__ int quad_at(int r, int q) { return r * 512 + ((q ^ (r & 7)) << 4); }

template <int DT> __global__ void __launch_bounds__(kThreads, 1) small_kernel(OrthogonalizeArgs a, int width) {
    extern __shared__ unsigned char dynamic[];
    __shared__ uint64_t bars[2];
    __shared__ uint32_t tmem;
    __shared__ int aborted;
    __shared__ float shared[kThreads / 32];
    __shared__ __align__(16) float squares[4];
    __shared__ Beginning begin;
    __shared__ StepFactors factors[kMostSteps];
    unsigned char* x = dynamic + (1024 - tc::shared_address(dynamic) % 1024) % 1024;
    const int cols = width / 64;                                  // blocks of X
    unsigned char* gram = x + cols * kBlock;                      // A, then the polynomial; the sums on their way
    const int t = static_cast<int>(threadIdx.x), warp = t >> 5, lane = t & 31, quarter = warp & 3, half = warp >> 2;
    const int row = quarter * 32 + lane;                          // of this thread's sums
    const uint32_t blocks = gridDim.x, rank = blocks > 1 ? tc::cluster_rank() : 0u;
    const uint32_t done = tc::shared_address(bars), drained = done + 8;
    if (t == 0) {
        tc::barrier_init(done, 1), tc::barrier_init(drained, 1);
        aborted = 0;
        tc::barrier_init_fence();
    }
    if (warp == 0) tc::tmem_alloc<512, false>(&tmem);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t acc = tmem, mine = acc + (static_cast<uint32_t>(quarter) << 21);
    volatile int* abort_word = &aborted;
    pdl_wait();

    const bool tall = a.rows > a.cols;
    const int m = static_cast<int>(tall ? a.cols : a.rows), n = static_cast<int>(tall ? a.rows : a.cols);
    const int c0 = static_cast<int>(rank) * width, have = max(0, min(width, n - c0));
    const size_t from = blockIdx.y * a.gstride;
    // X, read once: a thread has up to 16 pieces of eight columns, four of a block,
    // in registers until the norm is known.
    float v[16][8];
    const auto row_of = [&](int i) { return tall ? t % 128 : t / 8 + 32 * (i % 4); };
    const auto piece_of = [&](int i) { return tall ? t / 128 + 2 * (i % 4) : t % 8; };
    constexpr int es = Elem<DT>::kSize;
    const char* base = static_cast<const char*>(a.g) + (from + (tall ? static_cast<size_t>(c0) * a.ldg : static_cast<size_t>(c0))) * es;
    if (tall) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = t % 128, c = i / 4 * 64 + 8 * piece_of(i) + j;
                v[i][j] = r < m && c < have ? load_elem<DT>(base, static_cast<size_t>(c) * a.ldg + r) : 0.0f;
            }
    } else if (((reinterpret_cast<uintptr_t>(a.g) | a.ldg * es | a.gstride * es) & 15) == 0 && have % 8 == 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = row_of(i), c = i / 4 * 64 + 8 * (t % 8);
            uint4 w[es / 2];
#pragma unroll
            for (int j = 0; j < es / 2; ++j) {
                w[j] = make_uint4(0u, 0u, 0u, 0u);
                if (r < m && c < have) w[j] = *reinterpret_cast<const uint4*>(base + (static_cast<size_t>(r) * a.ldg + c) * es + 16 * j);
            }
#pragma unroll
            for (int j = 0; j < es / 2; ++j) {
                Acc<DT> x4;
                acc_seed<DT>(x4, w[j]);
#pragma unroll
                for (int e = 0; e < Elem<DT>::kVE; ++e) v[i][Elem<DT>::kVE * j + e] = x4.v[e];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = row_of(i), c = i / 4 * 64 + 8 * (t % 8) + j;
                v[i][j] = r < m && c < have ? load_elem<DT>(base, static_cast<size_t>(r) * a.ldg + c) : 0.0f;
            }
    }
    Squares q;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < 4 * cols) {
            Squares eight;
#pragma unroll
            for (int j = 0; j < 8; ++j) eight.add(v[i][j]);
            q.add(eight);
        }
    const float big = block_sum(q.big, shared), mid = block_sum(q.mid, shared), small = block_sum(q.small, shared);
    if (t == 0) squares[0] = big, squares[1] = mid, squares[2] = small, squares[3] = 0.0f;
    __syncthreads();
    if (blocks > 1) tc::cluster_sync();
    if (warp == 0) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (lane < static_cast<int>(blocks)) v = tc::load_cluster(tc::place_in(tc::shared_address(squares), static_cast<uint32_t>(lane)));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            v.x = __fadd_rn(v.x, __shfl_xor_sync(0xFFFFFFFFu, v.x, d));
            v.y = __fadd_rn(v.y, __shfl_xor_sync(0xFFFFFFFFu, v.y, d));
            v.z = __fadd_rn(v.z, __shfl_xor_sync(0xFFFFFFFFu, v.z, d));
        }
        if (lane == 0) begin = beginning(v.x, v.y, v.z, a.eps);
    }
    __syncthreads();
    if (t == kThreads - 1) step_factors(a, begin, factors);
    const Beginning f0 = begin;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < 4 * cols) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = f0.of(v[i][j]);
            uint4 hi, lo;
            split8(v[i], hi, lo);
            unsigned char* to = x + i / 4 * kBlock + piece_at(row_of(i), piece_of(i));
            *reinterpret_cast<uint4*>(to) = hi;
            *reinterpret_cast<uint4*>(to + kHalfBlock) = lo;
        }

    // Products of 64 along k of 128 x N, into the accumulators at `to`; one thread.
    const auto products = [&](uint32_t to, uint32_t left, uint32_t right, uint32_t lead, uint32_t b_step, uint32_t instruction) {
        const auto operand_b = [&](uint32_t at) { return tc::operand(at, lead, 1024); };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            tc::mma_f16<false>(to, tc::operand(left + 32 * i, 0, 1024), operand_b(right + kHalfBlock + b_step * i), instruction, i != 0);
            tc::mma_f16<false>(to, tc::operand(left + kHalfBlock + 32 * i, 0, 1024), operand_b(right + b_step * i), instruction, true);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            tc::mma_f16<false>(to, tc::operand(left + 32 * i, 0, 1024), operand_b(right + b_step * i), instruction, true);
    };
    uint32_t phase = 0;
    bool ok = true;
    // What threads wrote before the products that read it, and the products before
    // the threads that use them.
    const auto begin_products = [&]() {
        tc::fence_async();
        tc::fence_before();
        __syncthreads();
        if (t == 0) tc::fence_after(), tc::fence_async();
    };
    const auto end_products = [&]() {
        if (t == 0) tc::mma_commit<false>(done);
        ok = tc::barrier_wait(done, phase, abort_word) && ok;
        phase ^= 1;
        tc::fence_after();
        __syncwarp();
    };
    const auto add_sums = [&](float (&s)[32], uint32_t column) {
        uint32_t v[32];
        tc::tmem_load(mine + column, v);
        tc::tmem_wait(v);
#pragma unroll
        for (int j = 0; j < 32; ++j) s[j] = __fadd_rn(s[j], __uint_as_float(v[j]));
    };
    const uint32_t x_at = tc::shared_address(x), gram_at = tc::shared_address(gram);
    const uint32_t square = tc::instruction_f16(128, 128, false, false), wide = tc::instruction_f16(128, width, false, true);
    const int chunks = m > 64 ? 2 : 1;                            // of 64 rows of k in A and X
    for (int step = 0; step < a.steps; ++step) {
        begin_products();
        const StepFactors f = factors[step];
        if (t == 0)
            for (int b = 0; b < cols; ++b) products(acc + 128 * b, x_at + b * kBlock, x_at + b * kBlock, 0, 32, square);
        end_products();
        float sums[2][32] = {};
        for (int b = 0; b < cols; ++b) {
            add_sums(sums[0], 128 * b + 64 * half);
            add_sums(sums[1], 128 * b + 64 * half + 32);
        }
        if (!ok) sums[0][0] = __uint_as_float(0x7FFFFFFFu);       // a wait ran out: NaN for the whole matrix
        if (blocks > 1) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float* s = &sums[i / 8][i % 8 * 4];
                *reinterpret_cast<float4*>(gram + quad_at(row, 16 * half + i)) = make_float4(s[0], s[1], s[2], s[3]);
            }
            tc::cluster_sync();
            // This block's share of the rows: pieces of eight columns, up to four a thread.
            const int pieces = 2048 / static_cast<int>(blocks), share = static_cast<int>(rank) * (128 / static_cast<int>(blocks));
            float v[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = t + kThreads * i;
                if (e < pieces) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
                    const int r = share + e / 16, p = e % 16;
                    for (uint32_t other = 0; other < blocks; ++other) {
                        const float4 u = tc::load_cluster(tc::place_in(gram_at + quad_at(r, 2 * p), other));
                        const float4 w = tc::load_cluster(tc::place_in(gram_at + quad_at(r, 2 * p + 1), other));
                        v[i][0] = __fadd_rn(v[i][0], u.x), v[i][1] = __fadd_rn(v[i][1], u.y);
                        v[i][2] = __fadd_rn(v[i][2], u.z), v[i][3] = __fadd_rn(v[i][3], u.w);
                        v[i][4] = __fadd_rn(v[i][4], w.x), v[i][5] = __fadd_rn(v[i][5], w.y);
                        v[i][6] = __fadd_rn(v[i][6], w.z), v[i][7] = __fadd_rn(v[i][7], w.w);
                    }
                }
            }
            tc::cluster_sync();                                   // all have read: A takes the sums' place
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = t + kThreads * i;
                if (e < pieces) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] = __fmul_rn(v[i][j], f.gram);
                    uint4 hi, lo;
                    split8(v[i], hi, lo);
                    const int r = share + e / 16, p = e % 16;
                    const uint32_t to = gram_at + static_cast<uint32_t>(p / 8 * static_cast<int>(kBlock) + piece_at(r, p % 8));
                    for (uint32_t other = 0; other < blocks; ++other) {
                        store_cluster(tc::place_in(to, other), hi);
                        store_cluster(tc::place_in(to + static_cast<uint32_t>(kHalfBlock), other), lo);
                    }
                }
            }
            tc::fence_async();
            tc::cluster_sync();
        } else {
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                float* s = &sums[p / 4][p % 4 * 8];
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = __fmul_rn(s[j], f.gram);
                uint4 hi, lo;
                split8(s, hi, lo);
                unsigned char* to = gram + half * kBlock + piece_at(row, p);
                *reinterpret_cast<uint4*>(to) = hi;
                *reinterpret_cast<uint4*>(to + kHalfBlock) = lo;
            }
        }
        begin_products();
        if (t == 0)
            for (int b = 0; b < chunks; ++b) products(acc + 128 * b, gram_at + b * kBlock, gram_at + b * kBlock, 0, 32, square);
        end_products();
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int j = 0; j < 32; ++j) sums[g][j] = 0.0f;
        for (int b = 0; b < chunks; ++b) {
            add_sums(sums[0], 128 * b + 64 * half);
            add_sums(sums[1], 128 * b + 64 * half + 32);
        }
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            float* s = &sums[p / 4][p % 4 * 8];
            unsigned char* at = gram + half * kBlock + piece_at(row, p);
            const uint4 h = *reinterpret_cast<const uint4*>(at), l = *reinterpret_cast<const uint4*>(at + kHalfBlock);
            const uint32_t hs[4] = {h.x, h.y, h.z, h.w}, ls[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float u[2], w[2];
                widen_word<SAR_FP16>(hs[j], u);
                widen_word<SAR_FP16>(ls[j], w);
                s[2 * j] = __fmaf_rn(f.square, s[2 * j], __fmul_rn(f.linear, __fadd_rn(u[0], w[0])));
                s[2 * j + 1] = __fmaf_rn(f.square, s[2 * j + 1], __fmul_rn(f.linear, __fadd_rn(u[1], w[1])));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (half * 64 + 8 * p + j == row && row < m) s[j] = __fadd_rn(s[j], f.diagonal);
            uint4 hi, lo;
            split8(s, hi, lo);
            *reinterpret_cast<uint4*>(at) = hi;
            *reinterpret_cast<uint4*>(at + kHalfBlock) = lo;
        }
        begin_products();
        if (t == 0)
            for (int b = 0; b < chunks; ++b)
                products(acc + kColumns * b, gram_at + b * kBlock, x_at + b * (kHalfBlock / 2), kBlock, 2048, wide);
        end_products();
        const bool last = step + 1 == a.steps;
        const int failed = last ? __syncthreads_or(!ok) : 0;      // and the polynomial's place is free
        for (int g = 0; g < cols; ++g) {
            float s[32] = {};
            const int c = half * (width / 2) + 32 * g;            // of this block
            for (int b = 0; b < chunks; ++b) add_sums(s, kColumns * b + c);
            if (!last) {
#pragma unroll
                for (int p = 0; p < 4; ++p) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[8 * p + j] = __fmul_rn(f.apply, s[8 * p + j]);
                    uint4 hi, lo;
                    split8(s + 8 * p, hi, lo);
                    unsigned char* to = x + c / 64 * kBlock + piece_at(row, c % 64 / 8 + p);
                    *reinterpret_cast<uint4*>(to) = hi;
                    *reinterpret_cast<uint4*>(to + kHalfBlock) = lo;
                }
                continue;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j)
                s[j] = failed ? __uint_as_float(0x7FFFFFFFu) : __fmul_rn(__fmul_rn(__fmul_rn(s[j], f.first), f.second), f.third);
            const size_t to = blockIdx.y * a.ostride;
            if (tall) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (row < m && c + j < have)
                        store_elem<DT>(a.out, to + static_cast<size_t>(c0 + c + j) * a.ldo + static_cast<size_t>(row), s[j]);
                continue;
            }
            float* stage = reinterpret_cast<float*>(gram) + warp * 1024;        // 32 x 32, so that rows leave in lines
#pragma unroll
            for (int p = 0; p < 8; ++p)
                *reinterpret_cast<float4*>(stage + lane * 32 + ((p ^ (lane & 7)) << 2)) =
                    make_float4(s[4 * p], s[4 * p + 1], s[4 * p + 2], s[4 * p + 3]);
            __syncwarp();
#pragma unroll 8
            for (int r = 0; r < 32; ++r)
                if (quarter * 32 + r < m && c + lane < have)
                    store_elem<DT>(a.out, to + static_cast<size_t>(quarter * 32 + r) * a.ldo + static_cast<size_t>(c0 + c + lane),
                                   stage[r * 32 + ((((lane >> 2) ^ (r & 7)) << 2) | (lane & 3))]);
            __syncwarp();
        }
    }
    if (t == 0 && aborted != 0) {                                 // products in flight
        tc::mma_commit<false>(drained);
        tc::barrier_wait(drained, 0, nullptr);
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after();
        tc::tmem_free<512, false>(acc);
    }
}

template <int DT> cudaError_t launch(const OrthogonalizeArgs& a, cudaStream_t s) {
    static std::atomic<bool> allowed[kDevices], clusters[kDevices];
    const size_t n = std::max(a.rows, a.cols);
    const int blocks = blocks_of(n);
    const size_t width = (n + static_cast<size_t>(blocks) * 64 - 1) / (static_cast<size_t>(blocks) * 64) * 64;
    const auto kernel = small_kernel<DT>;
    cudaError_t e = allow_smem(kernel, std::max(kAlone, 1024 + (kColumns / 64 + 2) * kBlock), allowed);
    if (e != cudaSuccess) return e;
    if (blocks > 8) {                                             // more than is portable, once per device
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
        if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
        if (!clusters[dev].load(std::memory_order_acquire)) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            clusters[dev].store(true, std::memory_order_release);
        }
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(blocks), attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(a.batch));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = std::max(blocks > 1 ? kAlone : 0, 1024 + (width / 64 + 2) * kBlock);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, static_cast<int>(width));
}

}  // namespace

bool orthogonalize_small_fits(size_t rows, size_t cols) {
    return std::min(rows, cols) <= 128 && std::max(rows, cols) <= static_cast<size_t>(kMostBlocks) * kColumns;
}

cudaError_t launch_orthogonalize_small(sar_dtype dt, const OrthogonalizeArgs& a, cudaStream_t s) {
    switch (dt) {
    case SAR_BF16: return launch<SAR_BF16>(a, s);
    case SAR_FP16: return launch<SAR_FP16>(a, s);
    default: return launch<SAR_FP32>(a, s);
    }
}

}  // namespace sar
