// experts.cu -- tokens' rows dispatched to their experts' segments, combined
// again, and the combine's gradient.
//
// All three read or write topk scattered rows for each token's row, and are
// bound by HBM: whole rows move in granules of up to 16 bytes, a thread owns
// one granule of a token's row at a time and has the topk rows' accesses (kJ at
// a time) in flight together.  A token's own row is read once for every eight
// choices by the dispatch and for every four by the gradient; the kernels that
// take one choice at a time read it for each, from L1 or L2 after the first.
//
// Measured (GB300, copy rate 6.78 TB/s), 16384 x 8 x 4096 bf16: dispatch 181 us
// (98% of the copy rate: it scatters, so that x is read once, where gathering by
// place would read each row topk times), combine 171 us (104%); combine's
// gradient 8192 x 4 x 8192 fp16 176 us (101%).  Small: dispatch of 32 x 8 rows of
// 2048 bf16 2.0 us, combine's gradient 512 x 2 x 1024 fp32 2.7 us.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "sar_device.cuh"
#include "sar_internal.h"

namespace sar {
namespace {

constexpr int kBlock = 256;

// Granules: GB bytes moved by one access, as 32-bit words.
template <int GB> struct Granule { uint32_t w[GB < 4 ? 1 : GB / 4]; };

template <int GB> __device__ __forceinline__ Granule<GB> load(const void* base, size_t byte) {
    const char* p = static_cast<const char*>(base) + byte;
    Granule<GB> g;
    if constexpr (GB == 16) {
        const uint4 v = ld_stream_ordered(reinterpret_cast<const uint4*>(p));
        g.w[0] = v.x, g.w[1] = v.y, g.w[2] = v.z, g.w[3] = v.w;
    } else if constexpr (GB == 8) {
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(g.w[0]), "=r"(g.w[1]) : "l"(p) : "memory");
    } else if constexpr (GB == 4) {
        asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(g.w[0]) : "l"(p) : "memory");
    } else if constexpr (GB == 2) {
        g.w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
        g.w[0] = *reinterpret_cast<const uint8_t*>(p);
    }
    return g;
}

template <int GB> __device__ __forceinline__ void store(void* base, size_t byte, const Granule<GB>& g) {
    char* p = static_cast<char*>(base) + byte;
    if constexpr (GB == 16) {
        st_stream(reinterpret_cast<uint4*>(p), make_uint4(g.w[0], g.w[1], g.w[2], g.w[3]));
    } else if constexpr (GB == 8) {
        asm volatile("st.global.L1::no_allocate.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(g.w[0]), "r"(g.w[1]) : "memory");
    } else if constexpr (GB == 4) {
        asm volatile("st.global.L1::no_allocate.u32 [%0], %1;" ::"l"(p), "r"(g.w[0]) : "memory");
    } else if constexpr (GB == 2) {
        *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(g.w[0]);
    } else {
        *reinterpret_cast<uint8_t*>(p) = static_cast<uint8_t>(g.w[0]);
    }
}

// Elements of a granule in binary32, and back.  A 2-byte granule holds one
// element in the low half.
template <int DT, int GB> struct Elements { static constexpr int kN = GB / Elem<DT>::kSize; };

template <int DT, int GB> __device__ __forceinline__ void widen(const Granule<GB>& g, float* x) {
    if constexpr (GB < 4) {
        float two[2];
        widen_word<DT>(g.w[0], two);
        x[0] = two[0];
    } else {
#pragma unroll
        for (int i = 0; i < GB / 4; ++i) widen_word<DT>(g.w[i], x + i * PerWord<DT>::kN);
    }
}

template <int DT, int GB> __device__ __forceinline__ Granule<GB> narrow(const float* x) {
    Granule<GB> g;
    if constexpr (GB < 4) {
        const float two[2] = {x[0], 0.0f};
        g.w[0] = narrow_word<DT>(two);
    } else {
#pragma unroll
        for (int i = 0; i < GB / 4; ++i) g.w[i] = narrow_word<DT>(x + i * PerWord<DT>::kN);
    }
    return g;
}

// The place of slot j of token t, -1 where there is none.
__device__ __forceinline__ int place_of(const ExpertArgs& a, size_t t, int j) {
    if (j >= a.topk) return -1;
    const int p = a.position[t * a.topk + j];
    return static_cast<uint32_t>(p) < a.capacity ? p : -1;
}

// A block's threads over tokens and columns: TX threads (a power of two) for
// each of kBlock / TX tokens; gridDim.y shares a row's granules.
struct Shape {
    unsigned tx, granules;       // threads, granules per row
    unsigned token_blocks;       // blocks (x) of tokens
    unsigned pad_blocks;         // blocks before them, kPadShares for each expert
};

// Blocks that clear the padding of a segment.  They come first in the grid, so
// that theirs is not the last work of a small call.
constexpr unsigned kPadShares = 4;

// Clears a share of the padding rows of a segment.
template <int GB> __device__ void clear_padding(const ExpertArgs& a, const Shape& sh, unsigned block, size_t es) {
    const unsigned e = block / kPadShares;
    const int64_t from = static_cast<int64_t>(a.offsets[e]) + a.counts[e], end = a.offsets[e + 1];
    const int64_t first = from < 0 ? 0 : from;        // stays in the matrix whatever the arrays hold
    const int64_t last = end < static_cast<int64_t>(a.capacity) ? end : static_cast<int64_t>(a.capacity);
    Granule<GB> zero = {};
    for (int64_t p = first + block % kPadShares; p < last; p += kPadShares)
        for (unsigned v = blockIdx.y * blockDim.x + threadIdx.x; v < sh.granules; v += gridDim.y * blockDim.x)
            store<GB>(a.out, (static_cast<size_t>(p) * a.ldo) * es + static_cast<size_t>(v) * GB, zero);
}

constexpr int kJ = 8;

template <int GB>
__global__ void __launch_bounds__(kBlock) dispatch_kernel(ExpertArgs a, Shape sh, unsigned es) {
    pdl_wait();
    if (blockIdx.x < sh.pad_blocks) {
        clear_padding<GB>(a, sh, blockIdx.x, es);
        return;
    }
    const size_t t = static_cast<size_t>(blockIdx.x - sh.pad_blocks) * (blockDim.x / sh.tx) + threadIdx.x / sh.tx;
    if (t >= a.tokens) return;
    const unsigned first = blockIdx.y * sh.tx + threadIdx.x % sh.tx, step = gridDim.y * sh.tx;
    for (int j0 = 0; j0 < a.topk; j0 += kJ) {
        int p[kJ];
#pragma unroll
        for (int j = 0; j < kJ; ++j) p[j] = place_of(a, t, j0 + j);
        for (unsigned v = first; v < sh.granules; v += step) {
            const Granule<GB> g = load<GB>(a.tok, t * a.ldt * es + static_cast<size_t>(v) * GB);
#pragma unroll
            for (int j = 0; j < kJ; ++j)
                if (p[j] >= 0) store<GB>(a.out, static_cast<size_t>(p[j]) * a.ldo * es + static_cast<size_t>(v) * GB, g);
        }
    }
}

// Sums on pairs of elements (one instruction for two, each half rounded as the
// scalar one); a granule of one element uses one half.
template <int DT, int GB> struct Sums {
    static constexpr int kN = Elements<DT, GB>::kN, kPairs = (kN + 1) / 2;
    float2 v[kPairs];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int p = 0; p < kPairs; ++p) v[p] = make_float2(-0.0f, -0.0f);
    }
    // += x, or += w * x by one fused multiply-add.
    __device__ __forceinline__ void add(const Granule<GB>& g, float w, bool weighted) {
        float x[2 * kPairs];
        x[2 * kPairs - 1] = 0.0f;
        widen<DT, GB>(g, x);
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
            const float2 f = make_float2(x[2 * p], x[2 * p + 1]);
            v[p] = weighted ? __ffma2_rn(make_float2(w, w), f, v[p]) : __fadd2_rn(v[p], f);
        }
    }
    __device__ __forceinline__ Granule<GB> rounded(bool any) const {
        float x[2 * kPairs];
#pragma unroll
        for (int p = 0; p < kPairs; ++p) x[2 * p] = any ? v[p].x : 0.0f, x[2 * p + 1] = any ? v[p].y : 0.0f;
        return narrow<DT, GB>(x);
    }
};

// out = sum of w * row over the kept slots.  The sum starts from -0, the exact
// identity of the round-to-nearest add, so that one row is copied bit for bit.
// kOne: at most kJ slots a token, whose places and weights are read once, and
// rows within 2^32 granules of the first, so that a row's place is 32 bits (of
// 16384 x 8 x 4096 bf16: 192 us -> 171).  1024 threads an SM (64 registers): 768
// take 178 us, 1280 spill and take 193; four rows ahead instead of eight 182.
// Blocks of 128 leave less of the last round empty: 1003 x 6 x 1500 fp16 6.3 -> 5.0.
constexpr int kCombineBlock = 128;
template <int DT, int WDT, int GB, bool kOne>
__global__ void __launch_bounds__(kCombineBlock, 8) combine_kernel(ExpertArgs a, Shape sh) {
    using Offset = std::conditional_t<kOne, uint32_t, size_t>;          // in granules
    constexpr Offset kNone = static_cast<Offset>(-1);
    constexpr size_t es = Elem<DT>::kSize;
    pdl_wait();
    const size_t t = static_cast<size_t>(blockIdx.x) * (blockDim.x / sh.tx) + threadIdx.x / sh.tx;
    if (t >= a.tokens) return;
    const unsigned first = blockIdx.y * sh.tx + threadIdx.x % sh.tx, step = gridDim.y * sh.tx;
    const bool weighted = a.weights != nullptr;
    const Offset ld = static_cast<Offset>(a.ldi * es / GB);
    Offset row[kJ];
    float w[kJ];
    auto slots_from = [&](int j0) {
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const int p = place_of(a, t, j0 + j);
            row[j] = p >= 0 ? static_cast<Offset>(p) * ld : kNone;
            w[j] = weighted && p >= 0 ? load_elem<WDT>(a.weights, t * a.topk + j0 + j) : 0.0f;
        }
    };
    if (kOne) slots_from(0);
    // Small granules take two places at a time, for as many bytes in flight
    // (8192 x 8 x 4097 bf16 226 -> 144 us, 4098 111 -> 102; four spill).
    constexpr int kPlaces = kOne && GB <= 4 ? 2 : 1;
    for (unsigned v = first; v < sh.granules; v += kPlaces * step) {
        Sums<DT, GB> sum[kPlaces];
#pragma unroll
        for (int i = 0; i < kPlaces; ++i) sum[i].clear();
        bool any = false;
        for (int j0 = 0; j0 < (kOne ? 1 : a.topk); j0 += kJ) {
            if (!kOne) slots_from(j0);
            Granule<GB> g[kPlaces][kJ];
#pragma unroll
            for (int i = 0; i < kPlaces; ++i)
#pragma unroll
                for (int j = 0; j < kJ; ++j)
                    if (row[j] != kNone && (i == 0 || v + i * step < sh.granules))
                        g[i][j] = load<GB>(a.rows_in, static_cast<size_t>(static_cast<Offset>(row[j] + v + i * step)) * GB);
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                if (row[j] == kNone) continue;
                any = true;
#pragma unroll
                for (int i = 0; i < kPlaces; ++i)
                    if (i == 0 || v + i * step < sh.granules) sum[i].add(g[i][j], w[j], weighted);
            }
        }
#pragma unroll
        for (int i = 0; i < kPlaces; ++i)
            if (i == 0 || v + i * step < sh.granules)
                store<GB>(a.out, t * a.ldo * es + static_cast<size_t>(v + i * step) * GB, sum[i].rounded(any));
    }
}

// A block of the backward kernels: a token's TX threads, or eight tokens' warps.
template <int TX> constexpr int kTokenBlock = TX == 128 ? 128 : kBlock;

// drows = w * dout, dweights = <dout, row>.  TX threads (whole warps) have a
// token's row; gridDim.y shares the slots, J at a time.  The dot products are
// summed over the threads in a fixed order.
template <int DT, int WDT, int GB, int TX, int J>
__global__ void __launch_bounds__(kTokenBlock<TX>) combine_backward_kernel(ExpertArgs a, Shape sh) {
    constexpr int N = Elements<DT, GB>::kN, W = TX / 32;
    constexpr size_t es = Elem<DT>::kSize;
    __shared__ float red[W > 1 ? W : 1][J];
    pdl_wait();
    if (blockIdx.x < sh.pad_blocks) {
        clear_padding<GB>(a, sh, blockIdx.x, es);
        return;
    }
    const size_t t = static_cast<size_t>(blockIdx.x - sh.pad_blocks) * (kTokenBlock<TX> / TX) + threadIdx.x / TX;
    const unsigned x = threadIdx.x % TX;
    if (t >= a.tokens) return;                        // whole warps; with W > 1 never
    for (int j0 = blockIdx.y * J; j0 < a.topk; j0 += gridDim.y * J) {
        int p[J];
        float w[J], dot[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            p[j] = place_of(a, t, j0 + j);
            w[j] = p[j] >= 0 ? load_elem<WDT>(a.weights, t * a.topk + j0 + j) : 0.0f;
            dot[j] = 0.0f;
        }
        for (unsigned v = x; v < sh.granules; v += TX) {
            const size_t at = static_cast<size_t>(v) * GB;
            const Granule<GB> gd = load<GB>(a.tok, t * a.ldt * es + at);
            Granule<GB> g[J];
            if (a.dweights != nullptr) {
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (p[j] >= 0) g[j] = load<GB>(a.rows_in, static_cast<size_t>(p[j]) * a.ldi * es + at);
            }
            float d[N];
            widen<DT, GB>(gd, d);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (p[j] < 0) continue;
                float y[N];
                if (a.dweights != nullptr) {
                    widen<DT, GB>(g[j], y);
#pragma unroll
                    for (int e = 0; e < N; ++e) dot[j] = __fmaf_rn(d[e], y[e], dot[j]);
                }
#pragma unroll
                for (int e = 0; e < N; ++e) y[e] = __fmul_rn(w[j], d[e]);
                store<GB>(a.out, static_cast<size_t>(p[j]) * a.ldo * es + at, narrow<DT, GB>(y));
            }
        }
        if (a.dweights == nullptr) continue;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) dot[j] = __fadd_rn(dot[j], __shfl_xor_sync(0xFFFFFFFFu, dot[j], k));
        if (W == 1) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (x == 0 && j0 + j < a.topk) store_elem<WDT>(a.dweights, t * a.topk + j0 + j, dot[j]);
        } else {
            if ((x & 31) == 0) {
#pragma unroll
                for (int j = 0; j < J; ++j) red[x / 32][j] = dot[j];
            }
            __syncthreads();
            if (x < J && j0 + static_cast<int>(x) < a.topk) {
                float s = red[0][x];
                for (int k = 1; k < W; ++k) s = __fadd_rn(s, red[k][x]);
                store_elem<WDT>(a.dweights, t * a.topk + j0 + x, s);
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------------------
// Rows that do not start alike.  Where the addresses allow granules of 4 bytes
// or less (odd row lengths), the written row is taken in chunks of 16 bytes from
// a 16-byte boundary, and the bytes read for one come from two aligned vectors
// (the second is a neighbour lane's first, from L1) by funnel shifts.  The
// vectors may hold bytes of the rows beside the one read, never bytes outside
// the matrix: windows at its ends, and the chunks at a row's ends, go by
// element.  Measured against granules (us): dispatch 8192 x 8 x 4097 bf16 117 /
// 189, 16384 x 8 x 201 26 / 38; combine's gradient 326 / 388, 64 / 97.  The
// combine itself did not gain (198 / 144 and 47 / 28) and stays with granules.
// ---------------------------------------------------------------------------

// A matrix that is read; rows start at base + i * pitch bytes.
struct Source {
    const char* base;
    const char* end;             // one past its last element
    size_t pitch;
    __device__ __forceinline__ Source(const void* p, size_t rows, size_t ld, size_t cols, size_t es)
        : base(static_cast<const char*>(p)), end(base + ((rows - 1) * ld + cols) * es), pitch(ld * es) {}
};

__device__ __forceinline__ uint4 ld_cached(const char* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

template <typename Unit> __device__ __noinline__ uint4 gather16(const char* at) {
    constexpr int kPerWord = 4 / sizeof(Unit);
    const Unit* u = reinterpret_cast<const Unit*>(at);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = 0;
#pragma unroll
        for (int k = 0; k < kPerWord; ++k) w[i] |= static_cast<uint32_t>(u[i * kPerWord + k]) << (8 * sizeof(Unit) * k);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The vectors around the 16 bytes at `at`, all of them in one row of `src`; at
// the matrix's ends the bytes themselves.
struct Window {
    uint4 a, b;
    unsigned shift;

    template <typename Unit> __device__ __forceinline__ void load(const Source& src, const char* at) {
        shift = static_cast<unsigned>(reinterpret_cast<uintptr_t>(at)) & 15u;
        const char* low = at - shift;
        b = make_uint4(0, 0, 0, 0);
        if (low >= src.base && low + (shift != 0 ? 32 : 16) <= src.end) {
            a = ld_cached(low);
            if (shift != 0) b = ld_cached(low + 16);
        } else {
            a = gather16<Unit>(at);
            shift = 0;
        }
    }
    __device__ __forceinline__ uint4 bytes() const {
        uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (shift & 8u) {
#pragma unroll
            for (int i = 0; i < 6; ++i) x[i] = x[i + 2];
        }
        if (shift & 4u) {
#pragma unroll
            for (int i = 0; i < 5; ++i) x[i] = x[i + 1];
        }
        const unsigned bits = (shift & 3u) * 8;
        return make_uint4(__funnelshift_r(x[0], x[1], bits), __funnelshift_r(x[1], x[2], bits),
                          __funnelshift_r(x[2], x[3], bits), __funnelshift_r(x[3], x[4], bits));
    }
};

__device__ __forceinline__ Granule<16> granule(const uint4& v) {
    Granule<16> g;
    g.w[0] = v.x, g.w[1] = v.y, g.w[2] = v.z, g.w[3] = v.w;
    return g;
}

__device__ __forceinline__ unsigned phase_of(const void* p) {
    return static_cast<unsigned>(reinterpret_cast<uintptr_t>(p)) & 15u;
}

// Chunk u of a row written at `row` has the row's bytes u * 16 - phase ... + 15;
// sh.granules counts chunks, which a row has whatever its phase.
template <typename Unit>
__global__ void __launch_bounds__(kBlock) dispatch_shift_kernel(ExpertArgs a, Shape sh) {
    constexpr size_t es = sizeof(Unit);
    pdl_wait();
    if (blockIdx.x < sh.pad_blocks) {
        Shape by_unit = sh;
        by_unit.granules = static_cast<unsigned>(a.cols);
        clear_padding<es>(a, by_unit, blockIdx.x, es);
        return;
    }
    const size_t t = static_cast<size_t>(blockIdx.x - sh.pad_blocks) * (blockDim.x / sh.tx) + threadIdx.x / sh.tx;
    if (t >= a.tokens) return;
    const Source src(a.tok, a.tokens, a.ldt, a.cols, es);
    const char* from = src.base + t * src.pitch;
    const long long bytes = static_cast<long long>(a.cols * es);
    for (unsigned u = blockIdx.y * sh.tx + threadIdx.x % sh.tx; u < sh.granules; u += gridDim.y * sh.tx) {
        for (int j = 0; j < a.topk; ++j) {
            const int p = place_of(a, t, j);
            if (p < 0) continue;
            char* row = static_cast<char*>(a.out) + static_cast<size_t>(p) * a.ldo * es;
            const long long at = static_cast<long long>(u) * 16 - phase_of(row);
            if (at >= 0 && at + 16 <= bytes) {
                Window w;
                w.load<Unit>(src, from + at);
                st_stream(reinterpret_cast<uint4*>(row + at), w.bytes());
            } else {
                for (long long i = at < 0 ? 0 : at; i < at + 16 && i < bytes; i += es)
                    *reinterpret_cast<Unit*>(row + i) = *reinterpret_cast<const Unit*>(from + i);
            }
        }
    }
}

// 16-bit elements; the rows read and written start alike (or none are read); dout
// by windows.
template <int DT, int WDT, int TX>
__global__ void __launch_bounds__(kTokenBlock<TX>) combine_backward_shift_kernel(ExpertArgs a, Shape sh) {
    constexpr int N = Elements<DT, 16>::kN, W = TX / 32;
    constexpr size_t es = Elem<DT>::kSize;
    __shared__ float red[W > 1 ? W : 1];
    pdl_wait();
    if (blockIdx.x < sh.pad_blocks) {
        Shape by_unit = sh;
        by_unit.granules = static_cast<unsigned>(a.cols);
        clear_padding<es>(a, by_unit, blockIdx.x, es);
        return;
    }
    const size_t t = static_cast<size_t>(blockIdx.x - sh.pad_blocks) * (kTokenBlock<TX> / TX) + threadIdx.x / TX;
    const unsigned x = threadIdx.x % TX;
    if (t >= a.tokens) return;                        // whole warps; with W > 1 never
    const Source src(a.tok, a.tokens, a.ldt, a.cols, es);
    const char* from = src.base + t * src.pitch;
    const long long bytes = static_cast<long long>(a.cols * es);
    for (int j = blockIdx.y; j < a.topk; j += gridDim.y) {
        const size_t slot = t * a.topk + j;
        const int p = place_of(a, t, j);
        float dot = 0.0f;
        if (p >= 0) {
            const float w = load_elem<WDT>(a.weights, slot);
            char* to = static_cast<char*>(a.out) + static_cast<size_t>(p) * a.ldo * es;
            const char* row = static_cast<const char*>(a.rows_in) + static_cast<size_t>(p) * a.ldi * es;
            const unsigned phase = phase_of(to);
#pragma unroll 2
            for (unsigned u = x; u < sh.granules; u += TX) {
                const long long at = static_cast<long long>(u) * 16 - phase;
                if (at >= 0 && at + 16 <= bytes) {
                    Window win;
                    win.template load<uint16_t>(src, from + at);
                    float y[N], d[N];
                    if (a.dweights != nullptr) widen<DT, 16>(load<16>(row, static_cast<size_t>(at)), y);
                    widen<DT, 16>(granule(win.bytes()), d);
                    if (a.dweights != nullptr) {
#pragma unroll
                        for (int e = 0; e < N; ++e) dot = __fmaf_rn(d[e], y[e], dot);
                    }
#pragma unroll
                    for (int e = 0; e < N; ++e) d[e] = __fmul_rn(w, d[e]);
                    store<16>(to, static_cast<size_t>(at), narrow<DT, 16>(d));
                } else {
                    for (int e = 0; e < N; ++e) {
                        const long long i = at + e * static_cast<long long>(es);
                        if (i < 0 || i >= bytes) continue;
                        const float d = load_elem<DT>(from + i, 0);
                        if (a.dweights != nullptr) dot = __fmaf_rn(d, load_elem<DT>(row + i, 0), dot);
                        store_elem<DT>(to + i, 0, __fmul_rn(w, d));
                    }
                }
            }
        }
        if (a.dweights == nullptr) continue;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) dot = __fadd_rn(dot, __shfl_xor_sync(0xFFFFFFFFu, dot, k));
        if (W == 1) {
            if (x == 0) store_elem<WDT>(a.dweights, slot, dot);
        } else {
            if ((x & 31) == 0) red[x / 32] = dot;
            __syncthreads();
            if (x == 0) {
                float s = red[0];
                for (int k = 1; k < W; ++k) s = __fadd_rn(s, red[k]);
                store_elem<WDT>(a.dweights, slot, s);
            }
            __syncthreads();
        }
    }
}

// Largest granule (16, 8, 4, 2 or 1 bytes) that divides every address, leading
// dimension and the row's length.
unsigned granule_of(std::initializer_list<const void*> ptrs, std::initializer_list<size_t> lds, size_t cols, size_t es) {
    size_t bits = cols * es;
    for (const void* p : ptrs) bits |= reinterpret_cast<uintptr_t>(p);
    for (size_t ld : lds) bits |= ld * es;
    unsigned g = 16;
    while (bits % g != 0) g /= 2;
    return g;
}

// Threads per row: a power of two that covers the row's granules, up to the block;
// with `fit` a smaller one where that leaves less than 7/8 of the places (granules
// below 16 bytes, which are not bound by HBM: dispatch 8192 x 8 x 151 fp32 21.3 ->
// 13.5 us, 4096 x 8 x 1500 bf16 24.0 -> 22.3, but 600 fp32, 16 bytes, 28.6 -> 33.4).
Shape shape_of(const ExpertArgs& a, size_t granules, unsigned least, unsigned block, bool fit) {
    Shape sh;
    sh.tx = least;
    while (sh.tx < block && sh.tx < granules) sh.tx *= 2;
    const auto places = [&](size_t tx) { return (granules + tx - 1) / tx * tx; };
    for (unsigned tx = sh.tx / 2; fit && tx >= 32 && tx >= least; tx /= 2)
        if (8 * places(tx) < 7 * places(sh.tx)) sh.tx = tx;
    sh.granules = static_cast<unsigned>(granules);
    const size_t per = block / sh.tx;
    sh.token_blocks = static_cast<unsigned>((a.tokens + per - 1) / per);
    sh.pad_blocks = a.counts != nullptr ? kPadShares * a.experts : 0;
    return sh;
}

// Blocks (y) that share a token's row, one granule a thread, while the grid stays
// within kSpread blocks.  Combine, bf16 (us, kSpread 304 / 1216 / 4864): 300 x 4 x
// 4096 3.6 / 3.1 / 3.1, 600 x 4 x 4096 4.3 / 4.1 / 4.8, 1200 x 4 x 4096 7.1 / 7.2 / 9.1.
constexpr unsigned kSpread = 1216;
unsigned row_shares(const Shape& sh) {
    const unsigned most = (sh.granules + sh.tx - 1) / sh.tx, want = kSpread / std::min(sh.token_blocks, kSpread);
    return std::max(1u, std::min(want, most));
}

// Rows by shifted windows: granules of 2 bytes or less from `least` bytes a row
// on, of 4 bytes from `least4` on (the rows' ends go by element).  Dispatch, us,
// windows / granules: 8192 x 8 rows of 131 bf16 14.7 / 16.4, 251 18.5 / 18.9; 4
// bytes: 130 bf16 13.9 / 10.4, 250 17.7 / 12.8, 151 fp32 20 / 20, 4098 bf16 116 /
// 140.  Combine's gradient: 130 bf16 29.8 / 38.6, 4098 322 / 387.
bool by_windows(unsigned granule, size_t row_bytes, size_t least, size_t least4) {
    return granule <= 4 && row_bytes >= (granule == 4 ? least4 : least);
}

// Chunks of a row wherever it starts.
size_t chunks(size_t row_bytes) { return row_bytes / 16 + 2; }

// Threads of a dispatch block: 128 for few tokens (32 x 8 x 2048 bf16 1.9 us, 2.05
// with 256), else 256 (16384 x 8 x 4096 181 us, 184 with 128).
unsigned dispatch_block(const ExpertArgs& a) { return a.tokens <= 608 ? 128 : kBlock; }

template <typename Unit> cudaError_t dispatch_shift(const ExpertArgs& a, cudaStream_t s) {
    const unsigned block = dispatch_block(a);
    const Shape sh = shape_of(a, chunks(a.cols * sizeof(Unit)), 8, block, false);
    return launch_kernel(dispatch_shift_kernel<Unit>, dim3(sh.pad_blocks + sh.token_blocks, row_shares(sh)), dim3(block), s, a,
                         sh);
}

template <int GB> cudaError_t dispatch(const ExpertArgs& a, size_t es, cudaStream_t s) {
    const unsigned block = dispatch_block(a);
    const Shape sh = shape_of(a, a.cols * es / GB, 8, block, GB < 16);
    return launch_kernel(dispatch_kernel<GB>, dim3(sh.pad_blocks + sh.token_blocks, row_shares(sh)), dim3(block), s, a, sh,
                         static_cast<unsigned>(es));
}

template <int DT, int WDT, int GB> cudaError_t combine(const ExpertArgs& a, cudaStream_t s) {
    const Shape sh = shape_of(a, a.cols * Elem<DT>::kSize / GB, 8, kCombineBlock, GB < 16);
    const dim3 grid(sh.token_blocks, row_shares(sh)), block(kCombineBlock);
    const size_t ld = a.ldi * Elem<DT>::kSize / GB;
    const bool near = a.capacity == 0 || ld < 0xFFFFFFFFu / a.capacity;       // a place and the row after it
    return a.topk <= kJ && near
               ? launch_kernel(combine_kernel<DT, WDT, GB, true>, grid, block, s, a, sh)
               : launch_kernel(combine_kernel<DT, WDT, GB, false>, grid, block, s, a, sh);
}

template <int DT, int WDT> cudaError_t combine_by_granule(const ExpertArgs& a, cudaStream_t s) {
    constexpr int es = Elem<DT>::kSize;
    const unsigned g = granule_of({a.rows_in, a.out}, {a.ldi, a.ldo}, a.cols, es);
    if (g == 16) return combine<DT, WDT, 16>(a, s);
    if (g == 8) return combine<DT, WDT, 8>(a, s);
    if (g == 4) return combine<DT, WDT, 4>(a, s);
    return combine<DT, WDT, es>(a, s);
}

// Whether the backward call has a block for each slot (else for four of a
// token's): while all threads are on the SMs together, about.  Measured (us, so /
// not): 512 x 2 x 1024 fp32 2.7 / 3.4, 600 x 4 x 1024 bf16 3.2 / 4.1, 1200 x 4 x
// 1024 4.0 / 4.3, 512 x 8 x 2048 7.0 / 6.4; longer rows 4 x 8 x 4096 2.7 / 2.9, 64
// x 8 x 4096 3.3 / 3.1, 600 x 4 x 4096 7.8 / 5.5.
bool slot_blocks(size_t slots, size_t granules) { return slots * granules <= (granules <= 256 ? 640000 : 160000); }

template <int DT, int WDT, int GB, int TX, int J> cudaError_t backward(const ExpertArgs& a, cudaStream_t s) {
    constexpr int block = kTokenBlock<TX>;
    Shape sh = shape_of(a, a.cols * Elem<DT>::kSize / GB, TX, block, false);
    sh.tx = TX;
    sh.token_blocks = static_cast<unsigned>((a.tokens + block / TX - 1) / (block / TX));
    const dim3 grid(sh.pad_blocks + sh.token_blocks, std::min((a.topk + J - 1) / J, 65535));
    return launch_kernel(combine_backward_kernel<DT, WDT, GB, TX, J>, grid, dim3(block), s, a, sh);
}

// Whether a warp has a token's row rather than a block of 256: up to 128 granules,
// and up to 511 if there are warps enough, unless the row fills 15/16 of the
// block's places (from 257 granules on, or granules of eight elements; a block does
// not pay for 256 of fewer).  Measured (us, warp / block): bf16
// 4096 x 8 rows of 160 granules 32.5 / 37.0, 230 49.2 / 46.7, 250 51.5 / 48.9, 255
// 52.8 / 50.0, 256 50.7 / 47.6, 257 54.6 / 53.7, 300 61.5 / 63.1, 375 80.1 / 76.5,
// 500 102.9 / 92.1, 511 107 / 95.5; 8192 x 8 rows 224 83 / 87, 240 90.8 / 90.6, 255
// 100 / 99, 256 97 / 94, 511 195 / 184.  fp32 8192 x 8 rows of 230 90 / 100, 255 99 /
// 107, 256 94 / 99, 375 143 / 157, 511 192 / 193; 4096 x 8 rows of 255 52.2 / 53.8,
// 511 100 / 95.5; but 4096 x 4 rows of 256 29.3 / 26.5.
constexpr size_t kWarpTokens = 2048;
bool warp_rows(size_t tokens, size_t granules, int elements) {
    const size_t places = (granules + kBlock - 1) / kBlock * kBlock;
    const bool filled = 16 * granules >= 15 * places && (granules > kBlock || elements == 8);
    return granules <= 128 || (granules < 2 * kBlock && tokens >= kWarpTokens && !filled);
}

template <int DT, int WDT, int GB> cudaError_t backward_by_shape(const ExpertArgs& a, cudaStream_t s) {
    const size_t granules = a.cols * Elem<DT>::kSize / GB;
    const bool few = slot_blocks(a.tokens * a.topk, granules);
    if (granules <= 128 && few) return backward<DT, WDT, GB, 32, 1>(a, s);
    if (few) return backward<DT, WDT, GB, 128, 1>(a, s);
    if (warp_rows(a.tokens, granules, Elements<DT, GB>::kN)) return backward<DT, WDT, GB, 32, 4>(a, s);
    return backward<DT, WDT, GB, 256, 4>(a, s);
}

template <int DT, int WDT, int TX> cudaError_t backward_shift(const ExpertArgs& a, cudaStream_t s) {
    constexpr int block = kTokenBlock<TX>;
    Shape sh = shape_of(a, chunks(a.cols * Elem<DT>::kSize), TX, block, false);
    sh.tx = TX;
    sh.token_blocks = static_cast<unsigned>((a.tokens + block / TX - 1) / (block / TX));
    const dim3 grid(sh.pad_blocks + sh.token_blocks, slot_blocks(a.tokens * a.topk, sh.granules) ? std::min(a.topk, 65535) : 1);
    return launch_kernel(combine_backward_shift_kernel<DT, WDT, TX>, grid, dim3(block), s, a, sh);
}

template <int DT, int WDT> cudaError_t backward_by_granule(const ExpertArgs& a, cudaStream_t s) {
    constexpr int es = Elem<DT>::kSize;
    const bool alike = a.dweights == nullptr ||
                       (((reinterpret_cast<uintptr_t>(a.rows_in) ^ reinterpret_cast<uintptr_t>(a.out)) & 15u) == 0 &&
                        (a.ldi * es - a.ldo * es) % 16 == 0);
    const unsigned g = a.dweights != nullptr ? granule_of({a.tok, a.rows_in, a.out}, {a.ldt, a.ldi, a.ldo}, a.cols, es)
                                             : granule_of({a.tok, a.out}, {a.ldt, a.ldo}, a.cols, es);
    if constexpr (es == 2) {                          // 4-byte elements are no faster by windows (127 / 124 us)
        if (alike && by_windows(g, a.cols * es, 256, 256))
            return a.cols * es <= 2048 ? backward_shift<DT, WDT, 32>(a, s) : backward_shift<DT, WDT, 256>(a, s);
    }
    if (g == 16) return backward_by_shape<DT, WDT, 16>(a, s);
    if (g == 8) return backward_by_shape<DT, WDT, 8>(a, s);
    return backward_by_shape<DT, WDT, es>(a, s);
}

}  // namespace

cudaError_t launch_expert_dispatch(size_t es, const ExpertArgs& a, cudaStream_t s) {
    const unsigned g = granule_of({a.tok, a.out}, {a.ldt, a.ldo}, a.cols, es);
    if (by_windows(g, a.cols * es, 256, 1024))
        return es == 1 ? dispatch_shift<uint8_t>(a, s) : (es == 2 ? dispatch_shift<uint16_t>(a, s) : dispatch_shift<uint32_t>(a, s));
    switch (g) {
    case 16: return dispatch<16>(a, es, s);
    case 8: return dispatch<8>(a, es, s);
    case 4: return dispatch<4>(a, es, s);
    case 2: return dispatch<2>(a, es, s);
    default: return dispatch<1>(a, es, s);
    }
}

cudaError_t launch_expert_combine(sar_dtype dt, sar_dtype wdt, const ExpertArgs& a, cudaStream_t s) {
    switch (dt) {
    case SAR_BF16:
        return wdt == SAR_FP32 ? combine_by_granule<SAR_BF16, SAR_FP32>(a, s) : combine_by_granule<SAR_BF16, SAR_BF16>(a, s);
    case SAR_FP16:
        return wdt == SAR_FP32 ? combine_by_granule<SAR_FP16, SAR_FP32>(a, s) : combine_by_granule<SAR_FP16, SAR_FP16>(a, s);
    case SAR_FP32: return combine_by_granule<SAR_FP32, SAR_FP32>(a, s);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_expert_combine_backward(sar_dtype dt, sar_dtype wdt, const ExpertArgs& a, cudaStream_t s) {
    switch (dt) {
    case SAR_BF16:
        return wdt == SAR_FP32 ? backward_by_granule<SAR_BF16, SAR_FP32>(a, s) : backward_by_granule<SAR_BF16, SAR_BF16>(a, s);
    case SAR_FP16:
        return wdt == SAR_FP32 ? backward_by_granule<SAR_FP16, SAR_FP32>(a, s) : backward_by_granule<SAR_FP16, SAR_FP16>(a, s);
    case SAR_FP32: return backward_by_granule<SAR_FP32, SAR_FP32>(a, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace sar
