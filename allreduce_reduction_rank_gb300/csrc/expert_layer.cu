// expert_layer.cu -- the whole expert layer of a few tokens, in two kernels:
//   in_kernel    h = act(w_in[e] . x) (* the second half)   for every slot
//   out_kernel   out = sum_j weight_j * (w_out[e] . h_j)     for every token
//
// A slot is one choice of one token.  The time is that of reading the chosen
// experts' weights once: 2 to 4 operations for a byte of them, so the tensor
// cores are not what matters, but how many bytes are on their way.  Warps load
// 16-byte pieces of the weights straight into registers, which are the left
// operand of mma.sync (16 rows of weights by 8 slots): a lane's piece holds
// consecutive k, and as the order of k within a product does not matter, the
// pieces are taken as they come, with the slots' values at the same k.  (On the
// 5th-generation tensor cores the weights would have to pass through shared
// memory for 128 rows at a time, too coarse to spread few experts evenly.)
//
// Both kernels first sort the slots by expert into items of up to 8, 16 or 32
// slots of one expert, each block for itself.  The sort is stable, so that every
// block has the same items.
//
// Precision: x and 16-bit weights are multiplied as they are, sums in binary32 (the
// tensor cores' are cut off, see kChain).  h is not rounded to the type: bf16 weights
// meet it as two bf16 numbers (16 bits), fp16 ones (whose range it may leave) as two tf32
// numbers (22 bits) with the weights widened exactly; binary32 values on both sides are
// two tf32 numbers each, all four products.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "sar_device.cuh"
#include "sar_internal.h"

namespace sar {
namespace {

constexpr int kSMs = 152;
constexpr int kMaxSlots = SAR_EXPERT_LAYER_MAX_SLOTS;

__device__ __forceinline__ float activate(float z, sar_activation act) {
    if (act == SAR_ACT_SILU) return __fdiv_rn(z, __fadd_rn(1.0f, expf(-z)));
    // erfc keeps its digits where 1 + erf would cancel
    if (act == SAR_ACT_GELU) return __fmul_rn(__fmul_rn(0.5f, z), erfcf(__fmul_rn(z, -0.70710678f)));
    return z <= 0.0f ? 0.0f : z;
}

// ---------------------------------------------------------------------------
// The slots by expert.
// ---------------------------------------------------------------------------
struct Items {
    int count;
    int16_t *expert, *first, *slots;     // of an item: its slots are sorted[first .. first + slots - 1]
    int16_t* sorted;
    int16_t *of, *item;                  // a slot's expert (-1: dropped); a kept slot's item
    int16_t* rank;                       // scratch: a slot's place among its expert's
    int* tally;                          // scratch: an expert's slots, then first item << 16 | first place
};
constexpr size_t kItemArrays = 6;
__host__ __device__ __forceinline__ size_t items_bytes(int slots) { return (kItemArrays * 2 * static_cast<size_t>(slots) + 15) / 16 * 16; }
__host__ __device__ __forceinline__ size_t scratch_bytes(int slots, int experts) { return 4 * static_cast<size_t>(experts) + 2 * static_cast<size_t>(slots); }

// items_bytes(slots) at `at`, scratch_bytes at `scratch` until sort_slots has returned.
__device__ __forceinline__ void place_items(Items& it, unsigned char* at, unsigned char* scratch, int slots, int experts) {
    int16_t* p = reinterpret_cast<int16_t*>(at);
    it.expert = p, it.first = p + slots, it.slots = p + 2 * slots, it.sorted = p + 3 * slots, it.of = p + 4 * slots, it.item = p + 5 * slots;
    it.tally = reinterpret_cast<int*>(scratch);
    it.rank = reinterpret_cast<int16_t*>(it.tally + experts);
}

__device__ __forceinline__ int expert_of(const LayerArgs& a, int id_bytes, int slot) {
    const int64_t e = id_bytes == 8 ? static_cast<const int64_t*>(a.ids)[slot] : static_cast<const int32_t*>(a.ids)[slot];
    return e >= 0 && e < a.experts ? static_cast<int>(e) : -1;
}

// The items of `have` slots at `start`, up to `per` slots each, from item `at` on.
__device__ __forceinline__ void write_items(Items& it, int expert, int start, int have, int at, int per) {
    for (int done = 0; done < have; done += per, ++at) {
        it.expert[at] = static_cast<int16_t>(expert);
        it.first[at] = static_cast<int16_t>(start + done);
        it.slots[at] = static_cast<int16_t>(min(per, have - done));
    }
}

__device__ __forceinline__ int scan_before(int v, int lane) {        // sum over the lanes below
    int s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int other = __shfl_up_sync(0xFFFFFFFFu, s, d);
        if (lane >= d) s += other;
    }
    return s - v;
}

// All threads of the block; it.count is the same for all of them afterwards.
__device__ void sort_slots(Items& it, int* count, const LayerArgs& a, int id_bytes, int per) {
    const int slots = a.tokens * a.topk, t = static_cast<int>(threadIdx.x), threads = static_cast<int>(blockDim.x), lane = t & 31;
    if (slots <= 32) {                                               // one warp, without a count for each expert
        if (t < 32) {
            const int e = lane < slots ? expert_of(a, id_bytes, lane) : -1;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, e), below = (1u << lane) - 1u;
            const bool leads = e >= 0 && (same & below) == 0u;
            const int have = leads ? __popc(same) : 0, items = (have + per - 1) / per;
            const int before = scan_before(items << 16 | have, lane);
            const int of = __shfl_sync(0xFFFFFFFFu, before, __ffs(same) - 1), rank = __popc(same & below);
            if (lane < slots) it.of[lane] = static_cast<int16_t>(e);
            if (e >= 0) {
                it.sorted[(of & 0xFFFF) + rank] = static_cast<int16_t>(lane);
                it.item[lane] = static_cast<int16_t>((of >> 16) + rank / per);
            }
            write_items(it, e, before & 0xFFFF, have, before >> 16, per);
            if (lane == 31) *count = (before >> 16) + items;
        }
        __syncthreads();
        it.count = *count;
        return;
    }
    for (int e = t; e < a.experts; e += threads) it.tally[e] = 0;
    __syncthreads();
    for (int s = t; s < slots; s += threads) it.of[s] = static_cast<int16_t>(expert_of(a, id_bytes, s));
    __syncthreads();
    if (t < 32) {
        for (int s0 = 0; s0 < slots; s0 += 32) {                     // places within an expert, in the order of the slots
            const int s = s0 + lane, e = s < slots ? it.of[s] : -1;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
            const int before = e >= 0 ? it.tally[e] : 0;
            __syncwarp();
            if (e >= 0) {
                it.rank[s] = static_cast<int16_t>(before + __popc(same & ((1u << lane) - 1u)));
                if (lane == __ffs(same) - 1) it.tally[e] = before + __popc(same);
            }
            __syncwarp();
        }
        int done = 0;                                                // items << 16 | slots so far
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
            const int e = e0 + lane, have = e < a.experts ? it.tally[e] : 0, v = ((have + per - 1) / per) << 16 | have;
            const int before = done + scan_before(v, lane);
            if (e < a.experts) it.tally[e] = before;
            write_items(it, e, before & 0xFFFF, have, before >> 16, per);
            done = __shfl_sync(0xFFFFFFFFu, before + v, 31);
        }
        if (lane == 0) *count = done >> 16;
    }
    __syncthreads();
    for (int s = t; s < slots; s += threads) {
        const int e = it.of[s];
        if (e < 0) continue;
        it.sorted[(it.tally[e] & 0xFFFF) + it.rank[s]] = static_cast<int16_t>(s);
        it.item[s] = static_cast<int16_t>((it.tally[e] >> 16) + it.rank[s] / per);
    }
    __syncthreads();
    it.count = *count;
}

// ---------------------------------------------------------------------------
// Operands.
// ---------------------------------------------------------------------------
// Weights are read once: not kept in L1.  A request covers 64 bytes of a row, and
// L2 fetches the 256 around them (32 x 8 of 128 experts: 186 -> 181 us).
__device__ __forceinline__ uint4 load_weights(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// How rows lie, and what is read of them:
// kWhole     whole pieces of 16 bytes on 16-byte boundaries, as they are;
// kElements  binary32 off the boundaries, element by element;
// kBlocks    16-bit types off the boundaries: the 16 rows of a left operand are taken
//            `cycle` rows apart, which start at one distance from a boundary.  Their
//            pieces are the blocks between the boundaries, and k begins that distance
//            before the row, for them and for the slots, so that the weights need one
//            load a piece and, at the ends, a mask.
// 17 x 3 of 20 experts of 1021 / 2015 bf16: 84 us, with each piece put together from two
// blocks 95; 17 x 3 of 20 of 1021 / 515 binary32: by elements 40 us, by blocks 74 (fewer and
// larger units of rows).
enum Layout { kWhole, kElements, kBlocks };

// Elements k .. of a row of n, those outside it zero (k may be negative); the block
// lies on a boundary and holds elements of the row.
template <int DT> __device__ __forceinline__ uint4 load_block(const char* row, int k, int n, bool there) {
    constexpr int es = Elem<DT>::kSize, ve = Elem<DT>::kVE, per = 4 / es;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (!there || k >= n || k <= -ve) return v;
    v = load_weights(row + static_cast<ptrdiff_t>(k) * es);
    if (k >= 0 && k + ve <= n) return v;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = k + i * per;
        if (per == 1) {
            w[i] = e >= 0 && e < n ? w[i] : 0u;
        } else {
            const uint32_t low = e >= 0 && e < n ? 0x0000FFFFu : 0u, high = e + 1 >= 0 && e + 1 < n ? 0xFFFF0000u : 0u;
            w[i] &= low | high;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements k .. of a row of x of n, whatever its alignment, those outside it zero.
template <int DT> __device__ __forceinline__ uint4 load_x(const char* row, int k, int n, bool there) {
    constexpr int es = Elem<DT>::kSize;
    uint32_t w[8] = {};
    if (es == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (there && k + i >= 0 && k + i < n) w[i] = reinterpret_cast<const uint32_t*>(row)[k + i];
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (!there || k >= n || k <= -8) return make_uint4(0u, 0u, 0u, 0u);
    if (k < 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i >= 0 && k + i < n) w[i >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[k + i]) << (16 * (i & 1));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // the two 16-byte blocks that hold the piece (only blocks that hold elements of the row)
    const char* p = row + static_cast<size_t>(k) * es;
    const int left = n - k, shift = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
    const uint4 v = *reinterpret_cast<const uint4*>(p - shift);
    uint4 next = make_uint4(0u, 0u, 0u, 0u);
    if (shift > 0 && left * es > 16 - shift) next = *reinterpret_cast<const uint4*>(p - shift + 16);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w, w[4] = next.x, w[5] = next.y, w[6] = next.z, w[7] = next.w;
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = shift & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t both = shift & 2 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
        const int rest = left - 2 * i;
        w[i] = rest <= 0 ? 0u : (rest == 1 ? both & 0xFFFFu : both);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Where the pieces are whole: zeros past the row's end.
template <bool kWeights> __device__ __forceinline__ uint4 load_whole(const char* p, bool there) {
    if (!there) return make_uint4(0u, 0u, 0u, 0u);
    return kWeights ? load_weights(p) : *reinterpret_cast<const uint4*>(p);
}

// A piece of the weights; `shift` is 0 but for kBlocks.
template <int DT, Layout L> __device__ __forceinline__ uint4 load_left(const char* row, int k, int n, bool there, int shift) {
    if (L == kWhole) return load_whole<true>(row + static_cast<size_t>(k) * Elem<DT>::kSize, there && k < n);
    if (L == kElements) return load_x<DT>(row, k, n, there);
    return load_block<DT>(row, k - shift, n, there);
}

template <int DT> __device__ __forceinline__ void mma_16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                         uint32_t b1) {
    if (DT == SAR_BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// v = hi + lo, both tf32 (11 bits): hi cut off, which cannot overflow, lo rounded.
// An infinity is all hi.
__device__ __forceinline__ void split_tf32(float v, uint32_t& hi, uint32_t& lo) {
    hi = __float_as_uint(v) & 0xFFFFE000u;
    const float rest = fabsf(v) <= 0x1.fffffep127f ? __fsub_rn(v, __uint_as_float(hi)) : 0.0f;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(rest));
    if (v != v) hi = 0x7FFFFFFFu;
}

// v0, v1 = hi + lo as pairs of bf16: hi cut off, lo rounded.
__device__ __forceinline__ void split_bf16(float v0, float v1, uint32_t& hi, uint32_t& lo) {
    const float most = 0x1.fffffep127f;
    const uint32_t u0 = __float_as_uint(v0), u1 = __float_as_uint(v1);
    hi = __byte_perm(v0 != v0 ? 0x7FFFFFFFu : u0, v1 != v1 ? 0x7FFFFFFFu : u1, 0x7632);
    const float r0 = fabsf(v0) <= most ? __fsub_rn(v0, __uint_as_float(u0 & 0xFFFF0000u)) : 0.0f;
    const float r1 = fabsf(v1) <= most ? __fsub_rn(v1, __uint_as_float(u1 & 0xFFFF0000u)) : 0.0f;
    const float r[2] = {r0, r1};
    lo = narrow_word<SAR_BF16>(r);
}

// A lane's piece of two rows of weights, ready to be multiplied by the slots of
// any number of items' eights.
template <int DT, bool kTwo> struct Left;       // kTwo: against h, in two numbers

template <int DT> struct Left<DT, false> {      // 16-bit weights against x
    uint32_t a[4], b[4];
    __device__ __forceinline__ void set(const uint4& p, const uint4& q) {
        a[0] = p.x, a[1] = p.y, a[2] = p.z, a[3] = p.w, b[0] = q.x, b[1] = q.y, b[2] = q.z, b[3] = q.w;
    }
    __device__ __forceinline__ void multiply(float (&d)[4], const uint4& x) const {
        mma_16<DT>(d, a[0], b[0], a[1], b[1], x.x, x.y);
        mma_16<DT>(d, a[2], b[2], a[3], b[3], x.z, x.w);
    }
};
// The slots' h in two numbers, split once for all rows.
template <int DT> struct Right;
template <> struct Right<SAR_BF16> {
    uint32_t hi[4], lo[4];
    __device__ __forceinline__ explicit Right(const float (&h)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) split_bf16(h[2 * i], h[2 * i + 1], hi[i], lo[i]);
    }
};
template <int N> struct RightTf32 {
    uint32_t hi[N], lo[N];
    __device__ __forceinline__ explicit RightTf32(const float (&h)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) split_tf32(h[i], hi[i], lo[i]);
    }
};
template <> struct Right<SAR_FP16> : RightTf32<8> { using RightTf32<8>::RightTf32; };
template <> struct Right<SAR_FP32> : RightTf32<4> { using RightTf32<4>::RightTf32; };

template <> struct Left<SAR_BF16, true> {
    uint32_t a[4], b[4];
    __device__ __forceinline__ void set(const uint4& p, const uint4& q) {
        a[0] = p.x, a[1] = p.y, a[2] = p.z, a[3] = p.w, b[0] = q.x, b[1] = q.y, b[2] = q.z, b[3] = q.w;
    }
    __device__ __forceinline__ void multiply(float (&d)[4], const Right<SAR_BF16>& h) const {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            mma_16<SAR_BF16>(d, a[i], b[i], a[i + 1], b[i + 1], h.lo[i], h.lo[i + 1]);
            mma_16<SAR_BF16>(d, a[i], b[i], a[i + 1], b[i + 1], h.hi[i], h.hi[i + 1]);
        }
    }
};
template <> struct Left<SAR_FP16, true> {
    float a[8], b[8];
    __device__ __forceinline__ void set(const uint4& p, const uint4& q) {
        widen_word<SAR_FP16>(p.x, a), widen_word<SAR_FP16>(p.y, a + 2), widen_word<SAR_FP16>(p.z, a + 4), widen_word<SAR_FP16>(p.w, a + 6);
        widen_word<SAR_FP16>(q.x, b), widen_word<SAR_FP16>(q.y, b + 2), widen_word<SAR_FP16>(q.z, b + 4), widen_word<SAR_FP16>(q.w, b + 6);
    }
    __device__ __forceinline__ void multiply(float (&d)[4], const Right<SAR_FP16>& h) const {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint32_t a0 = __float_as_uint(a[i]), a1 = __float_as_uint(b[i]), a2 = __float_as_uint(a[i + 1]), a3 = __float_as_uint(b[i + 1]);
            mma_tf32(d, a0, a1, a2, a3, h.lo[i], h.lo[i + 1]);
            mma_tf32(d, a0, a1, a2, a3, h.hi[i], h.hi[i + 1]);
        }
    }
};
struct LeftFp32 {
    uint32_t ah[4], al[4], bh[4], bl[4];
    __device__ __forceinline__ void set(const uint4& p, const uint4& q) {
        split_tf32(__uint_as_float(p.x), ah[0], al[0]), split_tf32(__uint_as_float(p.y), ah[1], al[1]);
        split_tf32(__uint_as_float(p.z), ah[2], al[2]), split_tf32(__uint_as_float(p.w), ah[3], al[3]);
        split_tf32(__uint_as_float(q.x), bh[0], bl[0]), split_tf32(__uint_as_float(q.y), bh[1], bl[1]);
        split_tf32(__uint_as_float(q.z), bh[2], bl[2]), split_tf32(__uint_as_float(q.w), bh[3], bl[3]);
    }
    // The tensor cores' sums lose their last bits towards zero, so that a chain of
    // them over all of k was off by up to 9e-6: every 16 of k end in a sum of their
    // own, the small products first, which is added rounded to nearest.
    __device__ __forceinline__ void multiply(float (&d)[4], const RightTf32<4>& x) const {
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            mma_tf32(s, al[i], bl[i], al[i + 1], bl[i + 1], x.lo[i], x.lo[i + 1]);
            mma_tf32(s, al[i], bl[i], al[i + 1], bl[i + 1], x.hi[i], x.hi[i + 1]);
            mma_tf32(s, ah[i], bh[i], ah[i + 1], bh[i + 1], x.lo[i], x.lo[i + 1]);
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2) mma_tf32(s, ah[i], bh[i], ah[i + 1], bh[i + 1], x.hi[i], x.hi[i + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = __fadd_rn(d[i], s[i]);
    }
    __device__ __forceinline__ void multiply(float (&d)[4], const uint4& x) const {
        const float v[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w)};
        multiply(d, RightTf32<4>(v));
    }
};
template <> struct Left<SAR_FP32, false> : LeftFp32 {};
template <> struct Left<SAR_FP32, true> : LeftFp32 {};

__host__ __device__ __forceinline__ int h_ld(int hidden) { return (hidden + 7) / 8 * 8; }

// The tensor cores' sums lose their last bits towards zero (by up to 4 * 2^-24 of them a
// product), so that a chain of them over a long k falls behind where its terms have one
// sign: 16-bit types by 1.7e-3 over 2^20 of k, by 7e-4 over 65536 on the way out.  A warp's
// chain ends after kChain products at most and joins its earlier ones, rounded to nearest,
// in the place in shared memory where its sums go at last.  In binary32, whose chains are
// 16 of k long (LeftFp32), so do kChain / 2 of their additions.  64 x 2 of 8 of 4096 / 8192
// fp16 395 -> 397 us, bf16 357 -> 375; 32 x 8 of 128 bf16 172 -> 173.
constexpr int kChain = 128;
// The steps of a chain; kTwo: against h.
template <int DT, bool kTwo> constexpr int kFold = kChain / (DT == SAR_FP32 || !kTwo ? 4 : DT == SAR_FP16 ? 16 : 8);

// ---------------------------------------------------------------------------
// h = act(w_in . x).  A block takes MT times 16 rows of an item's expert, its warps a
// share of k each.  Gated: of whole pieces, 8 rows and the 8 that belong to them,
// which meet in one lane's sums; of other rows (whose two kinds start at distances of
// their own) 16 and 16, which meet in the sums of two left operands.
// ---------------------------------------------------------------------------
constexpr int kInWarps = 4;
// Blocks of the grid for a SM, in turn where fewer fit: 10 of items of eight slots fit in
// 16 bits (48 registers), 8 in binary32 (62), four off the boundaries (113); of the others
// two to six.  With 3, 4, 5, 8, 10, 12 of eight slots (us): 32 x 8 of 128 bf16 263, 221, 202,
// 180, 173, 196, fp32 621, 541, 494, 470, 485, 466; 17 x 3 of 20 of 1021 / 2015 bf16 94, 80,
// 100, 83, 84, 85.  With 2, 3, 4, 6, 8, 10 of more: 64 x 2 of 8 bf16 493, 403, 372, 416, 375,
// 394; 24 x 2 of 8 of 2048 / 4096 fp32 245, 210, 240, 210, 210, 212; 40 x 2 of 8 of 1022 /
// 2014 fp16 86, 74, 63, 65, 65, 65.
template <int N8> constexpr int kInBlocks = N8 == 1 ? 10 : 8;

// Blocks of a SM that the registers have to leave room for, where the compiler would take
// more of them (16 bits, 32 slots: 136, and three blocks; 64 x 2 of 8 fp16 446 us, with room
// for four 397).  0: no such bound, which costs spills elsewhere (32 x 8 of 128 bf16 191 us
// with one block to leave room for, 216 with ten, 173 without).
template <int DT, Layout L, int N8> constexpr int kResident = L != kWhole || N8 == 1 ? 0 : DT == SAR_FP32 ? (N8 == 2 ? 3 : 2) : N8 == 2 ? 6 : 4;

template <int DT, Layout L, int N8, int MT>
__global__ void __launch_bounds__(kInWarps * 32, kResident<DT, L, N8>) in_kernel(LayerArgs a, int id_bytes, int row_tiles, int cycle) {
    static_assert(L != kBlocks || MT == 2, "gates and what they gate");
    constexpr bool blocks = L == kBlocks;
    constexpr int ve = Elem<DT>::kVE, es = Elem<DT>::kSize, step = 8 * ve;      // 128 bytes of a row
    extern __shared__ __align__(16) unsigned char dynamic[];
    __shared__ __align__(16) float parts[kInWarps][MT * N8][32][4];
    __shared__ int item_count;
    const int slots = a.tokens * a.topk;
    Items it;
    place_items(it, dynamic, dynamic + items_bytes(slots), slots, a.experts);
    pdl_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // out_kernel may sort its slots meanwhile
    sort_slots(it, &item_count, a, id_bytes, 8 * N8);
    const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31, g = lane >> 2, c = lane & 3;
    const int rows = a.gated ? 2 * a.hidden : a.hidden, ld = h_ld(a.hidden);
    // The place in h of row r of 16 of the m-th left operand of a tile.
    const auto place_of = [&](int tile, int m, int r) {
        if (!blocks) return a.gated ? (tile * MT + m) * 8 + r % 8 : (tile * MT + m) * 16 + r;
        return tile / cycle * (a.gated ? 16 : 32) * cycle + tile % cycle + cycle * (a.gated ? r : 16 * m + r);
    };
    const auto is_gated_by = [&](int m, int r) { return a.gated && (blocks ? m == 1 : r >= 8); };
    const size_t row_bytes = static_cast<size_t>(a.cols) * es;
    const int units = it.count * row_tiles;
    for (int unit = static_cast<int>(blockIdx.x); unit < units; unit += static_cast<int>(gridDim.x)) {
        const int item = unit / row_tiles, tile = unit % row_tiles, n = it.slots[item], first = it.first[item];
        const char* base = static_cast<const char*>(a.w_in) + static_cast<size_t>(it.expert[item]) * rows * row_bytes;
        const char* w[MT][2];
        bool there[MT][2];
        int shift[MT] = {}, most = 0;                                // elements from a boundary to the rows' start
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * i + g, at = place_of(tile, m, r);
                there[m][i] = at < a.hidden;
                w[m][i] = base + (static_cast<size_t>(is_gated_by(m, r) ? a.hidden : 0) + (there[m][i] ? at : 0)) * row_bytes;
            }
            if (blocks) {
                const int at = place_of(tile, m, 0);
                const char* row = base + (static_cast<size_t>(is_gated_by(m, 0) ? a.hidden : 0) + at) * row_bytes;
                shift[m] = at < a.hidden ? static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / es : 0;
                most = max(most, shift[m]);
            }
        }
        const char* x[N8];
#pragma unroll
        for (int j = 0; j < N8; ++j) {
            const int t = 8 * j + g < n ? it.sorted[first + 8 * j + g] / a.topk : 0;
            x[j] = static_cast<const char*>(a.x) + static_cast<size_t>(t) * a.ldx * es;
        }
        constexpr int U = MT == 1 && N8 < 4 && L == kWhole ? 2 : 1;         // steps whose loads are on their way together
        constexpr int xm = blocks ? MT : 1;                            // x at each left operand's k
        constexpr int stride = U * kInWarps * step, chain = kFold<DT, false> / U * stride;
        const int end = a.cols + most;
        for (int k1 = warp * step; k1 == warp * step || k1 < end; k1 += chain) {
            float acc[MT][N8][4] = {};
            for (int k0 = k1; k0 < min(end, k1 + chain); k0 += stride) {
                uint4 p[2 * U][MT][2], v[2 * U][xm][N8];
#pragma unroll
                for (int u = 0; u < 2 * U; ++u) {
                    const int k = k0 + (u >> 1) * kInWarps * step + (u & 1) * 4 * ve + c * ve;
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            p[u][m][i] = load_left<DT, L>(w[m][i], k, a.cols, there[m][i], shift[m]);
#pragma unroll
                    for (int m = 0; m < xm; ++m)
#pragma unroll
                        for (int j = 0; j < N8; ++j)
                            v[u][m][j] = L == kWhole ? load_whole<false>(x[j] + static_cast<size_t>(k) * es, 8 * j + g < n && k < a.cols)
                                                     : load_x<DT>(x[j], k - shift[m], a.cols, 8 * j + g < n);
                }
#pragma unroll
                for (int u = 0; u < 2 * U; ++u) {
                    Left<DT, false> l[MT];
#pragma unroll
                    for (int m = 0; m < MT; ++m) l[m].set(p[u][m][0], p[u][m][1]);
#pragma unroll
                    for (int j = 0; j < N8; ++j)
                        if (j == 0 || 8 * j < n) {
#pragma unroll
                            for (int m = 0; m < MT; ++m) l[m].multiply(acc[m][j], v[u][blocks ? m : 0][j]);
                        }
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < N8; ++j) {
                    float4* at = reinterpret_cast<float4*>(parts[warp][m * N8 + j][lane]);
                    const float(&v)[4] = acc[m][j];
                    float4 sum = make_float4(v[0], v[1], v[2], v[3]);
                    if (k1 > warp * step) {
                        const float4 had = *at;
                        sum = make_float4(__fadd_rn(had.x, v[0]), __fadd_rn(had.y, v[1]), __fadd_rn(had.z, v[2]), __fadd_rn(had.w, v[3]));
                    }
                    *at = sum;
                }
        }
        __syncthreads();
        const auto sums_of = [&](int m, int j, float (&z)[4]) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                z[q] = parts[0][m * N8 + j][lane][q];
#pragma unroll
                for (int v = 1; v < kInWarps; ++v) z[q] = __fadd_rn(z[q], parts[v][m * N8 + j][lane][q]);
            }
        };
        // z[0], z[1]: row g of the operand, slots 2 c and 2 c + 1 of the eight; z[2], z[3]: row g + 8.
        const auto write = [&](int j, int q, int at_row, float value) {
            const int at = 8 * j + 2 * c + q;
            if (at < n && at_row < ld)
                static_cast<float*>(a.workspace)[static_cast<size_t>(it.sorted[first + at]) * ld + at_row] = at_row < a.hidden ? value : 0.0f;
        };
        for (int i = warp; i < MT * N8; i += kInWarps) {
            const int j = i % N8, m = i / N8;
            if (8 * j >= n || (blocks && a.gated && m == 1)) continue;
            float z[4], with[4];
            sums_of(m, j, z);
            if (blocks && a.gated) sums_of(1, j, with);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float h0 = activate(z[q], a.activation);
                if (!blocks && a.gated) {
                    write(j, q, place_of(tile, m, g), __fmul_rn(h0, z[2 + q]));
                    continue;
                }
                const float h1 = activate(z[2 + q], a.activation);
                write(j, q, place_of(tile, m, g), a.gated ? __fmul_rn(h0, with[q]) : h0);
                write(j, q, place_of(tile, m, g + 8), a.gated ? __fmul_rn(h1, with[2 + q]) : h1);
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// out = sum of weight * (w_out . h).  A cluster of blocks takes MT times 16
// columns of the output for all items.  Its warps take an item's share of k at a
// time, whose sums stay in their block's shared memory until all are there; then
// they are added in the order of the choices.
// ---------------------------------------------------------------------------
constexpr int kOutWarps = 16;                                        // one block a SM
constexpr int kMostParts = 16;
constexpr int kMostCluster = 8;

// Shares of k for an item: the number with the least time of a warp, which is its
// units times their steps (and two steps' time to begin and end one), as far as
// the sums of all slots fit.
__host__ __device__ __forceinline__ int parts_that_fit(int slots, int mt) {
    const int fit = kMaxSlots / (slots * mt);
    return fit < 1 ? 1 : (fit > kMostParts ? kMostParts : fit);
}
__device__ __forceinline__ int k_parts(int items, int slots, int steps, int warps, int mt) {
    const int most = max(1, min(steps / 2, parts_that_fit(slots, mt)));
    int best = 1, least = 0x7FFFFFFF;
    for (int p = 1; p <= most; ++p) {
        const int time = (items * p + warps - 1) / warps * ((steps + p - 1) / p + 2);
        if (time < least) best = p, least = time;
    }
    return best;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float load_of_block(const float* p, int rank) {      // the same place in a block of the cluster
    uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at));
    return v;
}

template <int DT, int WDT, Layout L, int N8, int MT>
__global__ void __launch_bounds__(kOutWarps * 32, 1) out_kernel(LayerArgs a, int id_bytes, int cycle) {
    static_assert(L != kBlocks || MT == 1, "one distance");
    constexpr int ve = Elem<DT>::kVE, es = Elem<DT>::kSize, step = 8 * ve, width = 16 * MT;
    extern __shared__ __align__(16) unsigned char dynamic[];
    __shared__ int item_count;
    const int slots = a.tokens * a.topk;
    float* sums = reinterpret_cast<float*>(dynamic + items_bytes(slots));       // parts x slots x width; the sort's scratch before
    Items it;
    place_items(it, dynamic, dynamic + items_bytes(slots), slots, a.experts);
    if (a.hidden == 0) pdl_wait();                                   // no in_kernel, which would have waited for the ids
    sort_slots(it, &item_count, a, id_bytes, 8 * N8);
    const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31, g = lane >> 2, c = lane & 3;
    const int blocks = static_cast<int>(gridDim.y), rank = static_cast<int>(blockIdx.y);
    const int steps = (a.hidden + (L != kBlocks || a.hidden == 0 ? 0 : ve - 1) + step - 1) / step, ld = h_ld(a.hidden);
    const int parts = k_parts(it.count, slots, steps, kOutWarps * blocks, MT), units = it.count * parts;
    const int block = static_cast<int>(blockIdx.x), c0 = block * width;
    const auto column_of = [&](int r) { return L != kBlocks ? c0 + r : block / cycle * width * cycle + block % cycle + cycle * r; };
    const size_t row_bytes = static_cast<size_t>(a.hidden) * es;
    // The weights do not depend on in_kernel: a warp's first ones go to L2 while it
    // ends (the first two lines of 16 rows; 1 x 8 of 128 experts 25.6 -> 22.8 us).
    if (L == kWhole && rank + blocks * warp < units) {
        const int unit = rank + blocks * warp, r = c0 + (lane & 15), s = unit % parts + (lane >> 4) * parts;
        if (r < a.cols && s < steps)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(a.w_out) +
                                                       (static_cast<size_t>(it.expert[unit / parts]) * a.cols + r) * row_bytes +
                                                       static_cast<size_t>(s) * 128));
    }
    pdl_wait();
    for (int unit = rank + blocks * warp; unit < units; unit += blocks * kOutWarps) {
        const int item = unit / parts, part = unit % parts, n = it.slots[item], first = it.first[item];
        const char* base = static_cast<const char*>(a.w_out) + static_cast<size_t>(it.expert[item]) * a.cols * row_bytes;
        const char* w[MT][2];
        bool there[MT][2];
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m) {
            const int r = column_of(8 * m + g);
            there[m >> 1][m & 1] = r < a.cols;
            w[m >> 1][m & 1] = base + (r < a.cols ? r : 0) * row_bytes;
        }
        int shift = 0;                                               // elements from a boundary to the rows' start
        if (L == kBlocks && column_of(0) < a.cols)
            shift = static_cast<int>(reinterpret_cast<uintptr_t>(base + column_of(0) * row_bytes) & 15) / es;
        const float* h[N8];
#pragma unroll
        for (int j = 0; j < N8; ++j)
            h[j] = static_cast<const float*>(a.workspace) +
                   static_cast<size_t>(8 * j + g < n ? it.sorted[first + 8 * j + g] : 0) * ld;
        constexpr int U = MT == 1 && N8 == 1 && L == kWhole ? 2 : 1;
        const int stride = U * parts, chain = kFold<DT, true> / U * stride;
        for (int s1 = part; s1 == part || s1 < steps; s1 += chain) {
            float acc[MT][N8][4] = {};
            for (int s0 = s1; s0 < min(steps, s1 + chain); s0 += stride) {
                uint4 p[2 * U][MT][2];
                float v[2 * U][N8][ve];
#pragma unroll
                for (int u = 0; u < 2 * U; ++u) {
                    const int k = (s0 + (u >> 1) * parts) * step + (u & 1) * 4 * ve + c * ve;
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            p[u][m][i] = load_left<DT, L>(w[m][i], k, a.hidden, there[m][i], shift);
#pragma unroll
                    for (int j = 0; j < N8; ++j) {
                        const bool have = 8 * j + g < n;
                        if (L != kBlocks) {
#pragma unroll
                            for (int i = 0; i < ve; i += 4) {            // rows of h end in zeros
                                float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                                if (have && k + i < a.hidden) q = *reinterpret_cast<const float4*>(h[j] + k + i);
                                v[u][j][i] = q.x, v[u][j][i + 1] = q.y, v[u][j][i + 2] = q.z, v[u][j][i + 3] = q.w;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < ve; ++i) {
                                const int at = k - shift + i;
                                v[u][j][i] = have && at >= 0 && at < a.hidden ? h[j][at] : 0.0f;
                            }
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < 2 * U; ++u) {
                    Left<DT, true> l[MT];
#pragma unroll
                    for (int m = 0; m < MT; ++m) l[m].set(p[u][m][0], p[u][m][1]);
#pragma unroll
                    for (int j = 0; j < N8; ++j)
                        if (j == 0 || 8 * j < n) {
                            const Right<DT> r(v[u][j]);
#pragma unroll
                            for (int m = 0; m < MT; ++m) l[m].multiply(acc[m][j], r);
                        }
                }
            }
#pragma unroll
            for (int j = 0; j < N8; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (8 * j + 2 * c + i < n) {
                        float* t = sums + (static_cast<size_t>(part) * slots + it.sorted[first + 8 * j + 2 * c + i]) * width + g;
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const float v0 = acc[m][j][i], v1 = acc[m][j][2 + i];
                            t[16 * m] = s1 > part ? __fadd_rn(t[16 * m], v0) : v0;
                            t[16 * m + 8] = s1 > part ? __fadd_rn(t[16 * m + 8], v1) : v1;
                        }
                    }
        }
    }
    cluster_sync();
    const int threads = blocks * kOutWarps * 32;
    for (int i = rank * kOutWarps * 32 + static_cast<int>(threadIdx.x); i < a.tokens * width; i += threads) {
        const int t = i / width, col = i % width, column = column_of(col);
        if (column >= a.cols) continue;
        float total = 0.0f;
        for (int j = 0; j < a.topk; ++j) {
            const int slot = t * a.topk + j;
            if (it.of[slot] < 0 || a.hidden == 0) continue;          // no sum, whatever its weight
            const int unit = it.item[slot] * parts;
            float s = 0.0f;
            for (int q = 0; q < parts; ++q)
                s = __fadd_rn(s, load_of_block(sums + (static_cast<size_t>(q) * slots + slot) * width + col, (unit + q) % blocks));
            total = __fmaf_rn(a.weights != nullptr ? load_elem<WDT>(a.weights, static_cast<size_t>(slot)) : 1.0f, s, total);
        }
        store_elem<DT>(a.out, static_cast<size_t>(t) * a.ldo + static_cast<size_t>(column), total);
    }
    cluster_sync();                                                  // no block ends while another reads its sums
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------
template <typename... KArgs>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s, KArgs... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1, attr[1].val.clusterDim.y = grid.y, attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// After how many rows their distance from a 16-byte boundary comes again.
int cycle_of(size_t row_bytes) {
    int cycle = 1;
    while (row_bytes * static_cast<size_t>(cycle) % 16 != 0) cycle *= 2;
    return cycle;
}

bool whole(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && bytes % 16 == 0; }

template <int DT, Layout L, int N8, int MT> cudaError_t launch_in(int id_bytes, const LayerArgs& a, cudaStream_t s) {
    const int slots = a.tokens * a.topk, cycle = L != kBlocks ? 1 : cycle_of(static_cast<size_t>(a.cols) * Elem<DT>::kSize);
    const int per = L != kBlocks ? (a.gated ? 8 : 16) * MT : (a.gated ? 16 : 32) * cycle;
    const int row_tiles = (a.hidden + per - 1) / per * cycle;
    const size_t most = static_cast<size_t>(slots) * static_cast<size_t>(row_tiles);
    const unsigned grid = static_cast<unsigned>(std::min<size_t>(most, kSMs * kInBlocks<N8>));
    return launch_kernel_smem(in_kernel<DT, L, N8, MT>, dim3(grid), dim3(kInWarps * 32),
                              items_bytes(slots) + scratch_bytes(slots, a.experts), s, a, id_bytes, row_tiles, cycle);
}

template <int DT, int WDT, Layout L, int N8, int MT> cudaError_t launch_out(int id_bytes, const LayerArgs& a, cudaStream_t s) {
    static std::atomic<bool> allowed[kDevices];
    const auto out = out_kernel<DT, WDT, L, N8, MT>;
    const cudaError_t e = allow_smem(out, items_bytes(kMaxSlots) + static_cast<size_t>(kMaxSlots) * 64, allowed);
    if (e != cudaSuccess) return e;
    const int slots = a.tokens * a.topk, cycle = L != kBlocks ? 1 : cycle_of(static_cast<size_t>(a.hidden) * Elem<DT>::kSize);
    const int per = 16 * MT * cycle, tiles = (a.cols + per - 1) / per * cycle;
    int blocks = 1;                                                  // as many blocks as are there at once
    while (blocks < kMostCluster && tiles * blocks * 2 <= kSMs) blocks *= 2;
    const size_t sums = static_cast<size_t>(parts_that_fit(slots, MT)) * slots * MT * 64;
    return launch_cluster(out, dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(blocks)), kOutWarps * 32,
                          items_bytes(slots) + std::max(scratch_bytes(slots, a.experts), sums), s, a, id_bytes, cycle);
}

// Slots of an item, by the slots that an expert has on average (of all experts: the host
// does not know which ones are chosen; where all tokens choose few of many experts, items
// stay at 8 and an expert's weights are read again for every 8 of its tokens):
// 8 up to 4 an expert.  8 experts of 2048 / 4096 with 8, and with 16 slots an item (us):
//   3 an expert: bf16 74.9, 74.4; 4: bf16 74.3, 75.8, fp32 198, 194; 5: 81.8, 78.9, fp32
//   213, 200; 8: 102, 87.
// 32 from 11 on, in binary32 from 21 on, with two left operands that share the slots' side,
// on the way in (on the way out, whose h takes twice the registers, 16).  8 experts of 4096
// / 8192 with 16, and with 32: 11 an expert: bf16 355, 329, fp32 1048, 1160; 16: fp16 454,
//   395, fp32 1365, 1390; 24: fp32 1928, 1777.  Of 2048 / 768 an expert's weights pass
//   quickly and 32 cost up to 9% (bf16 14 an expert: 55, 60; 24: 66, 69; 32: 89, 84).
// Off the 16-byte boundaries 8 up to 6, then 16: 8 experts of 2046 / 4094 with 8, and with
//   16: 6 an expert: bf16 137, 143, fp16 140, 159, fp32 295, 299; 7: 162, 157, 165, 172,
//   337, 320; 8: 176, 163, 180, 178, 365, 332.
// On the way out two left operands as far as the sums of all slots fit (32 columns of 512).
template <int DT, int WDT> cudaError_t launch(int id_bytes, const LayerArgs& a, cudaStream_t s) {
    constexpr size_t es = Elem<DT>::kSize;
    constexpr Layout off = es == 4 ? kElements : kBlocks;
    constexpr int off_mt = es == 4 ? 1 : 2;
    const bool in_whole = whole(a.w_in, static_cast<size_t>(a.cols) * es) && whole(a.x, a.ldx * es);
    const bool out_whole = whole(a.w_out, static_cast<size_t>(a.hidden) * es);
    const int mean = a.tokens * a.topk / a.experts;                  // slots of an expert
    const int many = es == 4 ? 20 : 10, off_few = 6;
    if (a.hidden > 0) {
        cudaError_t e;
        if (!in_whole)
            e = mean <= off_few ? launch_in<DT, off, 1, off_mt>(id_bytes, a, s) : launch_in<DT, off, 2, off_mt>(id_bytes, a, s);
        else if (mean <= 4)
            e = launch_in<DT, kWhole, 1, 1>(id_bytes, a, s);
        else
            e = mean <= many ? launch_in<DT, kWhole, 2, 2>(id_bytes, a, s) : launch_in<DT, kWhole, 4, 2>(id_bytes, a, s);
        if (e != cudaSuccess) return e;
    }
    if (!out_whole) return mean <= off_few ? launch_out<DT, WDT, off, 1, 1>(id_bytes, a, s) : launch_out<DT, WDT, off, 2, 1>(id_bytes, a, s);
    if (mean <= 4) return launch_out<DT, WDT, kWhole, 1, 1>(id_bytes, a, s);
    if (a.tokens * a.topk <= kMaxSlots / 2) return launch_out<DT, WDT, kWhole, 2, 2>(id_bytes, a, s);
    return launch_out<DT, WDT, kWhole, 2, 1>(id_bytes, a, s);
}

}  // namespace

size_t expert_layer_workspace_bytes(size_t slots, size_t, size_t hidden) {
    return 16 + slots * static_cast<size_t>(h_ld(static_cast<int>(hidden))) * sizeof(float);
}

cudaError_t launch_expert_layer(sar_dtype dt, sar_dtype wdt, int id_bytes, const LayerArgs& a, cudaStream_t s) {
    switch (dt) {
    case SAR_BF16: return wdt == SAR_FP32 ? launch<SAR_BF16, SAR_FP32>(id_bytes, a, s) : launch<SAR_BF16, SAR_BF16>(id_bytes, a, s);
    case SAR_FP16: return wdt == SAR_FP32 ? launch<SAR_FP16, SAR_FP32>(id_bytes, a, s) : launch<SAR_FP16, SAR_FP16>(id_bytes, a, s);
    default: return launch<SAR_FP32, SAR_FP32>(id_bytes, a, s);
    }
}

}  // namespace sar
