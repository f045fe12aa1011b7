// layer_norm_ring.cuh -- the layer norm kernels for many rows.
//
// One block on each SM stays for many rows.  A row belongs to a group of whole
// warps, as few as cover it, which has a range of the rows and works on R of
// them at a time (a batch).  Thread t of the group's `tpr` has NV vectors of
// each row, vector i at 16-byte place i * tpr + t; it copies them into its own
// places of a ring of D batches in shared memory with cp.async, D - 1 batches
// ahead, and only itself reads them again.  So the copies need no barrier, 100 KB and more are in flight on
// each SM whatever the registers hold, and the parameters and the sums for
// their gradients stay in registers.  What a batch costs beside its elements,
// the sums over the threads and a barrier, is shared by its rows: the sums of R
// rows travel together, halving their number with each exchange between lanes.
//
// Measured (GB300, copy rate 6.78 TB/s): forward 16384 x 8192 bf16 84 us, 94% of
// the copy rate, bound by HBM; backward 32768 x 4096 fp16 117 us without the
// parameters' gradients (101%), 121 with; 8192 x 4096 36.0 us (82%: launches,
// the ring's first fill and its last batch are 3 us and the parameters' sums 4).
// Whole warps and groups leave lanes of a block idle at other widths, 8192 rows of
// bf16, forward / backward: 2880 columns (70% of the lanes) 64 / 67% of the copy
// rate, 4608 (56%) 67 / 72, 5120 (62%) 73 / 77, 6144 (75%) 82 / 83, 7168 (88%) 86 /
// 87, 8192 (all) 91 / 91, 12288 (75%) 82 / 84.
// Depth: backward D = 3 41.0 us, D = 2 38.8 (less to fill before the first row
// and to work off after the last load); forward NV = 2 D = 2 90.1, 3 84.5, 6
// 88.4.  R = 1 backward 41, and 128 registers with half the threads 42.  The loads
// alone, from registers with one row ahead, took 61 us backward and 126 forward.
//
// Rows need not start on 16-byte boundaries (kShift): where the matrices of a
// call do so alike, row r starts `shift` elements past a boundary, with a period
// of 1, 2, 4 or 8 rows.  A group takes rows of one residue only, so its threads
// keep their columns: place k holds columns k * VE - shift ... + VE - 1.  The
// vectors at a row's ends are copied whole, with bytes of the neighbouring row
// or gap that are masked when they are read; only the first row's start and the
// last row's end, where there may be no such bytes, are copied by element.
// That is done when the row is read, in a function of its own: inside the copies
// it held registers (8192 x 4085 bf16 backward 50.2 -> 45.3 us, 4096 x 12001 90.7
// -> 82.7, 16384 x 1021 34.0 -> 33.0; 32768 x 1021 fp32 67 -> 69).
// 32768 x 1021 fp32 backward 68 us (87%); bf16, forward / backward: 16384 x 1021 41 /
// 45% (1024: 71 / 73%), 65536 x 130 27 / 28%, 32768 x 321 28 / 30%, 8192 x 4099 36 /
// 48%, 8192 x 4085 58 / 64%, 4096 x 12001 47 / 52%.
#pragma once

#include "layer_norm.cuh"

namespace sar {
namespace norm {

// Most threads of a block: one vector a thread fits 64 registers, so 1024; more
// vectors run with half of that.  The places of a ring are this far apart.
template <int NV> constexpr int kRingThreads = NV == 1 ? 1024 : 512;

// cp.async of 16 bytes, or 16 zero bytes where `have` is false.
__device__ __forceinline__ void copy_async(uint4* dst, const void* src, bool have) {
    const int n = have ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A thread's place in its group's rows.
template <int DT, bool kShift> struct Place {
    static constexpr int VE = Elem<DT>::kVE, es = Elem<DT>::kSize;
    int t, tpr, shift, cols;
    unsigned flags;              // of vector i, from bit 4 i: some of it is in the row, all is, it has the row's start, end

    __device__ __forceinline__ Place(int t_, int tpr_, int shift_, int cols_, int vectors)
        : t(t_), tpr(tpr_), shift(shift_), cols(cols_), flags(0) {
        if (!kShift) return;
        for (int i = 0; i < vectors; ++i) {
            const int c = column(i);
            const bool start = c < 0, end = c < cols && c + VE > cols;
            flags |= ((c < cols ? 1u : 0u) | (c < cols && !start && !end ? 2u : 0u) | (start ? 4u : 0u) | (end ? 8u : 0u)) << (4 * i);
        }
    }
    // First column of vector i; element e of it is column + e.
    __device__ __forceinline__ int column(int i) const { return (i * tpr + t) * VE - (kShift ? shift : 0); }
    __device__ __forceinline__ bool has(int c) const { return c < cols && (!kShift || c >= 0); }
    // Some of the vector's elements are in the row; all are.
    __device__ __forceinline__ bool some(int i) const {
        return kShift ? (flags & (1u << (4 * i))) != 0 : column(i) < cols;
    }
    __device__ __forceinline__ bool whole(int i) const {
        return kShift ? (flags & (2u << (4 * i))) != 0 : column(i) < cols;
    }
    // Its byte in the row; a 16-byte boundary even where it is past the row.
    __device__ __forceinline__ int byte(int i) const { return (i * tpr + t) * 16 - (kShift ? shift * es : 0); }
};

// Copies a thread's part of one row into its places.  `edge`: the matrix's first
// row (4), whose start, or its last (8), whose end may have nothing beside it;
// those vectors become zeros here and are left to patch_row.
template <int DT, int NV, int BT, bool kShift>
__device__ __forceinline__ void copy_row(uint4* slots, const char* row, const Place<DT, kShift>& at, unsigned edge) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool have = at.some(i) && !(kShift && ((at.flags >> (4 * i)) & edge));
        copy_async(slots + i * BT + threadIdx.x, row + (at.some(i) ? at.byte(i) : at.byte(0) - at.t * 16), have);
    }
}

// Copies what copy_row left, element by element, once the thread's own copies
// of the batch have ended.
template <int DT, int NV, int BT, bool kShift>
__device__ __noinline__ void patch_row(uint4* slots, const char* row, const Place<DT, kShift>& at, unsigned edge) {
    constexpr int VE = Elem<DT>::kVE, es = Elem<DT>::kSize;
    for (int i = 0; i < NV; ++i) {
        if (!((at.flags >> (4 * i)) & edge)) continue;
        uint4* slot = slots + i * BT + threadIdx.x;
        const int c = at.column(i);
        for (int e = 0; e < VE; ++e) {
            if (!at.has(c + e)) continue;
            if (es == 2) reinterpret_cast<uint16_t*>(slot)[e] = reinterpret_cast<const uint16_t*>(row)[c + e];
            else reinterpret_cast<uint32_t*>(slot)[e] = reinterpret_cast<const uint32_t*>(row)[c + e];
        }
    }
}

// Which bits of vector i are in the row.
template <int DT, bool kShift> __device__ __forceinline__ uint4 bits_of(int i, const Place<DT, kShift>& at) {
    constexpr int N = PerWord<DT>::kN;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = at.column(i) + k * N;
        w[k] = at.has(c) ? (N == 2 ? 0xFFFFu : 0xFFFFFFFFu) : 0u;
        if (N == 2 && at.has(c + 1)) w[k] |= 0xFFFF0000u;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Vector i of a row in pairs, zeros where it is past the row's ends.  With one
// vector a thread its bits are kept in registers, else worked out where needed.
template <int DT, int NV, int BT, bool kShift>
__device__ __forceinline__ void read_vec(const uint4* slots, int i, const Place<DT, kShift>& at, const uint4& bits, float2* x) {
    uint4 v = slots[i * BT + threadIdx.x];
    constexpr bool kAlways = NV == 1 && Elem<DT>::kVE == 8;        // cheaper than the branch
    if (kShift && (kAlways || !at.whole(i))) {
        const uint4 m = NV == 1 ? bits : bits_of<DT, kShift>(i, at);
        v = make_uint4(v.x & m.x, v.y & m.y, v.z & m.z, v.w & m.w);
    }
    widen<DT>(v, x);
}

// Zeros in the pairs of vector i that are past the row's ends.
template <int DT> __device__ __forceinline__ void clear_outside(const uint4& bits, float2* x) {
    constexpr int P = Elem<DT>::kVE / 2;
    const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const uint32_t lo = PerWord<DT>::kN == 2 ? static_cast<uint32_t>(static_cast<int32_t>(w[p % 4] << 16) >> 16) : w[2 * p % 4];
        const uint32_t hi = PerWord<DT>::kN == 2 ? static_cast<uint32_t>(static_cast<int32_t>(w[p % 4]) >> 16) : w[(2 * p + 1) % 4];
        x[p].x = __uint_as_float(__float_as_uint(x[p].x) & lo);
        x[p].y = __uint_as_float(__float_as_uint(x[p].y) & hi);
    }
}

template <int DT, int NV, bool kShift>
__device__ __forceinline__ void write_vec(char* row, int i, const Place<DT, kShift>& at, const uint4& bits, const float2* x) {
    constexpr int VE = Elem<DT>::kVE, N = PerWord<DT>::kN;
    float f[VE];
#pragma unroll
    for (int p = 0; p < VE / 2; ++p) f[2 * p] = x[p].x, f[2 * p + 1] = x[p].y;
    char* to = row + at.byte(i);
    if (!kShift) {                                    // packed inside the branch: 36.0 us, before it 36.8 (backward 8192 x 4096)
        if (at.whole(i))
            st_stream(reinterpret_cast<uint4*>(to),
                      make_uint4(narrow_word<DT>(f), narrow_word<DT>(f + N), narrow_word<DT>(f + 2 * N), narrow_word<DT>(f + 3 * N)));
        return;
    }
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = narrow_word<DT>(f + k * N);
    if (at.whole(i)) {
        st_stream(reinterpret_cast<uint4*>(to), make_uint4(u[0], u[1], u[2], u[3]));
    } else if (at.some(i)) {                          // words where they are whole
        const uint4 m = NV == 1 ? bits : bits_of<DT, kShift>(i, at);
        const uint32_t have[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (have[k] == 0xFFFFFFFFu) reinterpret_cast<uint32_t*>(to)[k] = u[k];
            else if (have[k] == 0x0000FFFFu) reinterpret_cast<uint16_t*>(to)[2 * k] = static_cast<uint16_t>(u[k]);
            else if (have[k] == 0xFFFF0000u) reinterpret_cast<uint16_t*>(to)[2 * k + 1] = static_cast<uint16_t>(u[k] >> 16);
        }
    }
}

// A thread's values of a parameter of type fp32 or DT; `none` without one.
template <int DT, int NV, bool kShift>
__device__ __forceinline__ void read_param(const void* p, bool w32, const Place<DT, kShift>& at, float none, float2* x) {
    constexpr int VE = Elem<DT>::kVE;
#pragma unroll
    for (int k = 0; k < NV * VE / 2; ++k) {
        const int c = at.column(2 * k / VE) + 2 * k % VE;
        x[k] = pair(none);
        if (p != nullptr && at.has(c)) x[k].x = w32 ? static_cast<const float*>(p)[c] : load_elem<DT>(p, c);
        if (p != nullptr && at.has(c + 1)) x[k].y = w32 ? static_cast<const float*>(p)[c + 1] : load_elem<DT>(p, c + 1);
    }
}

// A barrier among the warps of group g (1 .. 15 of them where a group has several).
__device__ __forceinline__ void ring_sync(int g, int wpg) {
    asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(32 * wpg) : "memory");
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
#pragma unroll
    for (; bit > 0; bit >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, bit));
    return s;
}

// The rows of a group: first + i * period for i = begin .. end - 1.  Groups of
// one residue share its rows evenly, each a contiguous range of the i.
// (A row here is longer than 240 bytes, so their number fits 32 bits.)
struct Rows {
    unsigned residue, begin, end, period;
    unsigned first, last;        // the i of the matrix's first and last row, where the residue has them
    __device__ __forceinline__ Rows(size_t all, unsigned id, unsigned groups, unsigned period_) : period(period_) {
        const unsigned rows = static_cast<unsigned>(all);
        residue = id % period;
        const unsigned mine = rows > residue ? (rows - residue + period - 1) / period : 0;
        const unsigned n = groups / period, g = id / period, per = mine / n, more = mine % n;
        begin = per * g + (g < more ? g : more);
        end = begin + per + (g < more ? 1 : 0);
        first = residue == 0 ? 0 : 0xFFFFFFFFu;
        last = (rows - 1) % period == residue ? (rows - 1) / period : 0xFFFFFFFFu;
    }
    __device__ __forceinline__ size_t row(unsigned i) const { return residue + static_cast<size_t>(i) * period; }
    // Whether it is the matrix's first (4) or last (8) row.
    __device__ __forceinline__ unsigned edge(unsigned i) const { return (i == first ? 4u : 0u) | (i == last ? 8u : 0u); }
};

template <int DT, int NV, int R, int D, bool kShift, int WPG>
__global__ void __launch_bounds__(kRingThreads<NV>, 1)
ring_forward_kernel(NormArgs a, bool w32, float inv_n, Alignment al, int wpg_any) {
    const int wpg = WPG != 0 ? WPG : wpg_any;
    const bool alone = NV == 1 && wpg == 1;           // a row to a warp: at most 32 vectors
    constexpr int VE = Elem<DT>::kVE, P = VE / 2, BT = kRingThreads<NV>, L = 32 / R;
    const int G = blockDim.x / (32 * wpg);            // groups, of wpg warps each
    extern __shared__ uint4 ring[];                   // [D][R][NV][threads]
    __shared__ float4 red[2][BT / 32][R];
    const unsigned lane = threadIdx.x & 31;
    const int g = __shfl_sync(0xFFFFFFFFu, threadIdx.x / (32 * wpg), 0);        // the same for a warp
    const float n = static_cast<float>(a.cols);
    const Rows rows(a.rows, blockIdx.x * G + g, gridDim.x * G, kShift ? al.period : 1);
    const Place<DT, kShift> at(static_cast<int>(threadIdx.x) - g * 32 * wpg, 32 * wpg,
                                       static_cast<int>((al.start + rows.residue * al.step) % VE), static_cast<int>(a.cols), NV);
    const uint4 bits = bits_of<DT, kShift>(0, at);
    pdl_wait();
    // Rows are walked by pointers: the products would cost more than the copies.
    constexpr size_t es = Elem<DT>::kSize;
    const size_t pitch_x = rows.period * a.ldx * es, pitch_y = rows.period * a.ldy * es;
    const char* next_x = static_cast<const char*>(a.x) + rows.row(rows.begin) * a.ldx * es;
    char* now_y = static_cast<char*>(a.y) + rows.row(rows.begin) * a.ldy * es;
    unsigned ahead = rows.begin;                      // first row of the next batch to copy
    int slot = 0;                                     // its place in the ring
    auto copy_batch = [&] {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (ahead + j >= rows.end) continue;
            copy_row<DT, NV, BT, kShift>(ring + (slot * R + j) * NV * BT, next_x, at, rows.edge(ahead + j));
            next_x += pitch_x;
        }
        copy_commit();
        ahead += R;
        slot = slot + 1 == D ? 0 : slot + 1;
    };
#pragma unroll
    for (int d = 0; d < D - 1; ++d) copy_batch();
    float2 w[NV * P], b[NV * P];
    read_param<DT, NV, kShift>(a.weight, w32, at, 1.0f, w);
    read_param<DT, NV, kShift>(a.bias, w32, at, 0.0f, b);
    bool whole = true;                                // all of this thread's vectors
    int held = 0;                                     // elements of this thread, then of its warp
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        whole = whole && at.whole(i);
        const int c = at.column(i), first = c < 0 ? 0 : c, last = c + VE < at.cols ? c + VE : at.cols;
        held += last > first ? last - first : 0;
    }
    held = __reduce_add_sync(0xFFFFFFFFu, held);
    const float have = static_cast<float>(held), inv_have = held > 0 ? 1.0f / have : 0.0f;
    int now = 0;
    for (unsigned r = rows.begin, k = 0; r < rows.end; r += R, ++k) {
        copy_wait<D - 2>();
        copy_batch();                                 // into the place of the batch before this one
        uint4* from = ring + now * R * NV * BT;
        now = now + 1 == D ? 0 : now + 1;
        if (kShift) {
#pragma unroll
            for (int j = 0; j < R; ++j)
                if (r + j < rows.end && rows.edge(r + j) != 0)
                    patch_row<DT, NV, BT, kShift>(from + j * NV * BT,
                                                  static_cast<const char*>(a.x) + rows.row(r + j) * a.ldx * es, at,
                                                  rows.edge(r + j));
        }
        float s[R], m[R], q[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float2 s2 = pair(0.0f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 f[P];
                read_vec<DT, NV, BT, kShift>(from + j * NV * BT, i, at, bits, f);
#pragma unroll
                for (int p = 0; p < P; ++p) s2 = __fadd2_rn(s2, f[p]);
            }
            s[j] = __fadd_rn(s2.x, s2.y);
        }
        const float total = scatter_sum<R>(s);
        // One warp takes the deviations around the row's mean, several each around one near their own.
        const float near = alone ? quotient(total, n, inv_n) : __fmul_rn(total, inv_have);
#pragma unroll
        for (int j = 0; j < R; ++j) m[j] = __shfl_sync(0xFFFFFFFFu, near, j * L);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float2 q2 = pair(0.0f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 f[P];
                widen<DT>(from[(j * NV + i) * BT + threadIdx.x], f);
#pragma unroll
                for (int p = 0; p < P; ++p) f[p] = __fadd2_rn(f[p], pair(-m[j]));
                if (!whole) clear_outside<DT>(NV == 1 ? bits : bits_of<DT, kShift>(i, at), f);
#pragma unroll
                for (int p = 0; p < P; ++p) q2 = __ffma2_rn(f[p], f[p], q2);
            }
            q[j] = __fadd_rn(q2.x, q2.y);
        }
        const float squares = scatter_sum<R>(q);
        float mean, rstd;                             // of row lane % R, or lane / L with one warp
        if (alone) {
            mean = near;
            rstd = rsqrtf(__fmaf_rn(squares, inv_n, a.eps));
        } else {
            float4(&all)[BT / 32][R] = red[k & 1];
            if (lane % L == 0) all[threadIdx.x / 32][lane / L] = make_float4(total, squares, near, have);
            ring_sync(g, wpg);
            constexpr int T = BT / 32 / L > 0 ? BT / 32 / L : 1;      // a lane's warps: lane / R, + L, ...
            float4 p[T];
            float sum = 0.0f, sq = 0.0f;
#pragma unroll
            for (int i = 0; i < T; ++i) {
                const int from_warp = lane / R + i * L;
                p[i] = from_warp < wpg ? all[g * wpg + from_warp][lane % R] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                sum = __fadd_rn(sum, p[i].x);
            }
#pragma unroll
            for (int d = R; d < 32; d <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xFFFFFFFFu, sum, d));
            mean = quotient(sum, n, inv_n);
#pragma unroll
            for (int i = 0; i < T; ++i) sq = __fadd_rn(sq, around(p[i], mean));
#pragma unroll
            for (int d = R; d < 32; d <<= 1) sq = __fadd_rn(sq, __shfl_xor_sync(0xFFFFFFFFu, sq, d));
            rstd = rsqrtf(__fmaf_rn(not_below_zero(sq), inv_n, a.eps));
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const float mj = __shfl_sync(0xFFFFFFFFu, mean, alone ? j * L : j);
            const float rj = __shfl_sync(0xFFFFFFFFu, rstd, alone ? j * L : j);
            if (r + j >= rows.end) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 f[P];
                widen<DT>(from[(j * NV + i) * BT + threadIdx.x], f);
#pragma unroll
                for (int p = 0; p < P; ++p)
                    f[p] = __ffma2_rn(__fmul2_rn(__fadd2_rn(f[p], pair(-mj)), pair(rj)), w[i * P + p], b[i * P + p]);
                write_vec<DT, NV, kShift>(now_y, i, at, bits, f);
            }
            now_y += pitch_y;
            if (at.t == 0) {
                const size_t row = rows.row(r + j);
                if (a.mean != nullptr) a.mean[row] = mj;
                if (a.rstd != nullptr) a.rstd[row] = rj;
            }
        }
    }
    copy_wait<0>();
}

// The sums over a group of N values per thread, in every thread of it.
template <int BT, int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float (*red)[N], int g, int wpg) {
    constexpr int L = 32 / N;
    const unsigned lane = threadIdx.x & 31;
    float s = scatter_sum<N>(v);
    if (wpg == 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, s, i * L);
        return;
    }
    if (lane % L == 0) red[threadIdx.x / 32][lane / L] = s;
    ring_sync(g, wpg);
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < (BT / 32 + L - 1) / L; ++i) {
        const int from = lane / N + i * L;
        if (from < wpg) s = __fadd_rn(s, red[g * wpg + from][lane % N]);
    }
#pragma unroll
    for (int d = N; d < 32; d <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, d));
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, s, i);
}

// A thread's sum of g h over its places in the row, from the ring (x, then dy;
// its first place is column c0) and the parameter, in the order of the pairs.
template <int DT, int NV, int BT>
__device__ __noinline__ float sum_in_row(const uint4* slots, const void* weight, bool w32, int c0, int tpr, int cols,
                                         float minus_mean, float rstd) {
    constexpr int VE = Elem<DT>::kVE;
    float even = 0.0f, odd = 0.0f;
    for (int i = 0; i < NV; ++i) {
        for (int e = 0; e < VE; ++e) {
            const int c = c0 + i * tpr * VE + e;
            if (c < 0 || c >= cols) continue;
            const float h = __fmul_rn(__fadd_rn(load_elem<DT>(slots + i * BT + threadIdx.x, e), minus_mean), rstd);
            const float dh = __fmul_rn(load_elem<DT>(slots + (NV + i) * BT + threadIdx.x, e), h);
            const float w = weight == nullptr ? 1.0f : (w32 ? static_cast<const float*>(weight)[c] : load_elem<DT>(weight, c));
            if (e % 2 == 0) even = __fmaf_rn(dh, w, even);
            else odd = __fmaf_rn(dh, w, odd);
        }
    }
    return __fadd_rn(even, odd);
}

template <int DT, int NV, int R, int D, bool kShift, int WPG>
__global__ void __launch_bounds__(kRingThreads<NV>, 1)
ring_backward_kernel(NormGradArgs a, bool w32, float inv_n, Alignment al, int wpg_any) {
    const int wpg = WPG != 0 ? WPG : wpg_any;
    constexpr int VE = Elem<DT>::kVE, P = VE / 2, BT = kRingThreads<NV>;
    const int G = blockDim.x / (32 * wpg);            // groups, of wpg warps each
    // x - mean and dy of a batch are kept for dx where the registers hold them,
    // else read from the ring again.
    constexpr bool kHold = NV == 1 && VE == 4;
    constexpr int HP = kHold ? P : 1;
    extern __shared__ uint4 ring[];                   // [D][R][x, dy][NV][threads]
    __shared__ float red[2][BT / 32][2 * R];
    const int g = __shfl_sync(0xFFFFFFFFu, threadIdx.x / (32 * wpg), 0);        // the same for a warp
    const Rows rows(a.rows, blockIdx.x * G + g, gridDim.x * G, kShift ? al.period : 1);
    const Place<DT, kShift> at(static_cast<int>(threadIdx.x) - g * 32 * wpg, 32 * wpg,
                                       static_cast<int>((al.start + rows.residue * al.step) % VE), static_cast<int>(a.cols), NV);
    const uint4 bits = bits_of<DT, kShift>(0, at);
    pdl_wait();
    constexpr size_t es = Elem<DT>::kSize;
    const size_t pitch_x = rows.period * a.ldx * es, pitch_dy = rows.period * a.lddy * es, pitch_dx = rows.period * a.lddx * es;
    const char* next_x = static_cast<const char*>(a.x) + rows.row(rows.begin) * a.ldx * es;
    const char* next_dy = static_cast<const char*>(a.dy) + rows.row(rows.begin) * a.lddy * es;
    char* now_dx = static_cast<char*>(a.dx) + rows.row(rows.begin) * a.lddx * es;
    unsigned ahead = rows.begin;
    int slot = 0;
    auto copy_batch = [&] {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (ahead + j >= rows.end) continue;
            const unsigned edge = rows.edge(ahead + j);
            uint4* to = ring + (slot * R + j) * 2 * NV * BT;
            copy_row<DT, NV, BT, kShift>(to, next_x, at, edge);
            copy_row<DT, NV, BT, kShift>(to + NV * BT, next_dy, at, edge);
            next_x += pitch_x, next_dy += pitch_dy;
        }
        copy_commit();
        ahead += R;
        slot = slot + 1 == D ? 0 : slot + 1;
    };
#pragma unroll
    for (int d = 0; d < D - 1; ++d) copy_batch();
    float2 w[NV * P], dw[NV * P], db[NV * P];
    read_param<DT, NV, kShift>(a.weight, w32, at, 1.0f, w);
#pragma unroll
    for (int p = 0; p < NV * P; ++p) dw[p] = db[p] = pair(0.0f);
    float mean[R], rstd[R];
    const float* next_mean = a.mean + rows.row(rows.begin);
    const float* next_rstd = a.rstd + rows.row(rows.begin);
    auto statistics = [&](unsigned r) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            mean[j] = r + j < rows.end ? next_mean[j * rows.period] : 0.0f;
            rstd[j] = r + j < rows.end ? next_rstd[j * rows.period] : 0.0f;
        }
        next_mean += R * rows.period, next_rstd += R * rows.period;
    };
    statistics(rows.begin);
    int now = 0;
    for (unsigned r = rows.begin, k = 0; r < rows.end; r += R, ++k) {
        copy_wait<D - 2>();
        copy_batch();                                 // into the place of the batch before this one
        uint4* from = ring + now * R * 2 * NV * BT;
        now = now + 1 == D ? 0 : now + 1;
        if (kShift) {
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const unsigned edge = r + j < rows.end ? rows.edge(r + j) : 0u;
                if (edge == 0) continue;
                const size_t row = rows.row(r + j);
                patch_row<DT, NV, BT, kShift>(from + 2 * j * NV * BT, static_cast<const char*>(a.x) + row * a.ldx * es, at, edge);
                patch_row<DT, NV, BT, kShift>(from + (2 * j + 1) * NV * BT, static_cast<const char*>(a.dy) + row * a.lddy * es,
                                              at, edge);
            }
        }
        float v[2 * R], rs[R], mj[R];
        float2 dev[R][HP], up[R][HP];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float2 s2 = pair(0.0f), q2 = pair(0.0f);
            rs[j] = rstd[j], mj[j] = -mean[j];
            // One vector a thread: its bits are at hand to mask with.  With more, which
            // have no registers for it, the thread's sum is taken again.
            const bool past = kShift && past_range<DT>(mj[j], rs[j]);
            if (r + j < rows.end) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float2 f[P], d[P];
                    read_vec<DT, NV, BT, kShift>(from + (j * 2) * NV * BT, i, at, bits, f);
                    read_vec<DT, NV, BT, kShift>(from + (j * 2 + 1) * NV * BT, i, at, bits, d);
                    const float m = kShift || at.some(i) ? mj[j] : 0.0f;        // whole vectors past the end: 0 - 0
#pragma unroll
                    for (int p = 0; p < P; ++p) f[p] = __fadd2_rn(f[p], pair(m));
                    if (NV == 1 && past) clear_outside<DT>(bits, f);
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const int c = i * P + p;
                        if (kHold) dev[j][p % HP] = f[p], up[j][p % HP] = d[p];
                        const float2 dh = __fmul2_rn(d[p], __fmul2_rn(f[p], pair(rs[j])));     // dy h
                        dw[c] = __fadd2_rn(dw[c], dh);
                        db[c] = __fadd2_rn(db[c], d[p]);
                        s2 = __ffma2_rn(d[p], w[c], s2);
                        q2 = __ffma2_rn(dh, w[c], q2);
                    }
                }
            }
            v[2 * j] = __fadd_rn(s2.x, s2.y);
            v[2 * j + 1] = __fadd_rn(q2.x, q2.y);
            if (NV > 1 && past)
                v[2 * j + 1] = sum_in_row<DT, NV, BT>(from + j * 2 * NV * BT, a.weight, w32, at.column(0), at.tpr, at.cols, mj[j], rs[j]);
        }
        statistics(r + R);
        group_sums<BT, 2 * R>(v, red[k & 1], g, wpg);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (r + j >= rows.end) continue;
            // dx = rstd (g - mean(g) - (x - mean) (rstd mean(g h))); rstd^2 could leave binary32's range.
            const float c0 = -__fmul_rn(v[2 * j], inv_n);
            const float c1 = -__fmul_rn(rs[j], __fmul_rn(v[2 * j + 1], inv_n));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 f[P], d[P];
                if (kHold) {
#pragma unroll
                    for (int p = 0; p < P; ++p) f[p] = dev[j][p % HP], d[p] = up[j][p % HP];
                } else {
                    widen<DT>(from[(j * 2 * NV + i) * BT + threadIdx.x], f);
                    widen<DT>(from[(j * 2 * NV + NV + i) * BT + threadIdx.x], d);
#pragma unroll
                    for (int p = 0; p < P; ++p) f[p] = __fadd2_rn(f[p], pair(mj[j]));
                }
#pragma unroll
                for (int p = 0; p < P; ++p)
                    f[p] = __fmul2_rn(__ffma2_rn(f[p], pair(c1), __ffma2_rn(d[p], w[i * P + p], pair(c0))), pair(rs[j]));
                write_vec<DT, NV, kShift>(now_dx, i, at, bits, f);
            }
            now_dx += pitch_dx;
        }
    }
    copy_wait<0>();
    if (a.dweight == nullptr && a.dbias == nullptr) return;
    // The groups' sums, added in order; through shared memory, so that they
    // leave in whole sectors.
    const unsigned cols = static_cast<unsigned>(a.cols);
    float* out = a.partial + static_cast<size_t>(blockIdx.x) * 2 * cols;
    float* sums = reinterpret_cast<float*>(ring);     // [G][2][cols]
    __syncthreads();
    if (kShift) {
#pragma unroll
        for (int e = 0; e < NV * VE; ++e) {
            const int c = at.column(e / VE) + e % VE;
            if (at.has(c)) {
                sums[g * 2 * cols + c] = e % 2 ? dw[e / 2].y : dw[e / 2].x;
                sums[(g * 2 + 1) * cols + c] = e % 2 ? db[e / 2].y : db[e / 2].x;
            }
        }
    } else {                                          // four columns at a time: single ones would meet in the banks
#pragma unroll
        for (int p = 0; p < NV * P; p += 2) {
            const int c = at.column(2 * p / VE) + 2 * p % VE;
            if (at.some(2 * p / VE)) {
                *reinterpret_cast<float4*>(sums + g * 2 * cols + c) = make_float4(dw[p].x, dw[p].y, dw[p + 1].x, dw[p + 1].y);
                *reinterpret_cast<float4*>(sums + (g * 2 + 1) * cols + c) = make_float4(db[p].x, db[p].y, db[p + 1].x, db[p + 1].y);
            }
        }
    }
    __syncthreads();
    for (unsigned c = threadIdx.x; c < 2 * cols; c += blockDim.x) {
        float v = sums[c];
        for (int p = 1; p < G; ++p) v = __fadd_rn(v, sums[p * 2 * cols + c]);
        out[c] = v;
    }
}

template <int DT, int NV, int R, int D, bool kShift, int WPG>
cudaError_t ring_launch_as(const NormArgs& a, bool w32, size_t vecs, const Alignment& al, cudaStream_t s) {
    static std::atomic<bool> allowed[kDevices];
    constexpr size_t smem = static_cast<size_t>(D) * R * NV * kRingThreads<NV> * 16;
    const cudaError_t e = allow_smem(ring_forward_kernel<DT, NV, R, D, kShift, WPG>, smem, allowed);
    if (e != cudaSuccess) return e;
    const RingSplit split = ring_split(vecs, NV);
    return launch_kernel_smem(ring_forward_kernel<DT, NV, R, D, kShift, WPG>, dim3(kSMs), dim3(split.groups * split.warps * 32), smem,
                              s, a, w32, 1.0f / static_cast<float>(a.cols), al, split.warps);
}

template <int DT, int NV, int R, int D, bool kShift, int WPG>
cudaError_t ring_launch_as(const NormGradArgs& a, bool w32, size_t vecs, const Alignment& al, cudaStream_t s) {
    static std::atomic<bool> allowed[kDevices];
    constexpr size_t smem = static_cast<size_t>(D) * R * 2 * NV * kRingThreads<NV> * 16;
    const cudaError_t e = allow_smem(ring_backward_kernel<DT, NV, R, D, kShift, WPG>, smem, allowed);
    if (e != cudaSuccess) return e;
    const RingSplit split = ring_split(vecs, NV);
    return launch_kernel_smem(ring_backward_kernel<DT, NV, R, D, kShift, WPG>, dim3(kSMs), dim3(split.groups * split.warps * 32), smem,
                              s, a, w32, 1.0f / static_cast<float>(a.cols), al, split.warps);
}

// Groups of 4, 8 or 16 warps, known when compiled, keep more in registers and
// skip the rest of the loops over warps (8192 x 4096 fp16 backward without the
// parameters' gradients: 35.5 us, 37.8 with the number known at run time).
template <int DT, int NV, int R, int D, bool kShift, class Args>
cudaError_t ring_launch(const Args& a, bool w32, size_t vecs, const Alignment& al, cudaStream_t s) {
    if constexpr (NV == 1) {
        switch (ring_split(vecs, NV).warps) {
        case 4: return ring_launch_as<DT, NV, R, D, kShift, 4>(a, w32, vecs, al, s);
        case 8: return ring_launch_as<DT, NV, R, D, kShift, 8>(a, w32, vecs, al, s);
        case 16: return ring_launch_as<DT, NV, R, D, kShift, 16>(a, w32, vecs, al, s);
        default: break;
        }
    } else if (ring_split(vecs, NV).warps == 16) {
        return ring_launch_as<DT, NV, R, D, kShift, 16>(a, w32, vecs, al, s);
    }
    return ring_launch_as<DT, NV, R, D, kShift, 0>(a, w32, vecs, al, s);
}

// `vecs` places a row, at most kRingVecs.
template <int DT, bool kShift> cudaError_t ring_any(const NormArgs& a, bool w32, size_t vecs, const Alignment& al, cudaStream_t s) {
    switch (ring_vectors(vecs)) {
    case 1: return ring_launch<DT, 1, 2, 3, kShift>(a, w32, vecs, al, s);
    case 2: return ring_launch<DT, 2, 2, 3, kShift>(a, w32, vecs, al, s);
    default: return ring_launch<DT, 4, 1, 6, kShift>(a, w32, vecs, al, s);
    }
}

template <int DT, bool kShift>
cudaError_t ring_any(const NormGradArgs& a, bool w32, size_t vecs, const Alignment& al, cudaStream_t s) {
    switch (ring_vectors(vecs)) {
    case 1: return ring_launch<DT, 1, 2, 2, kShift>(a, w32, vecs, al, s);
    case 2: return ring_launch<DT, 2, 2, 2, kShift>(a, w32, vecs, al, s);
    default: return ring_launch<DT, 4, 1, 2, kShift>(a, w32, vecs, al, s);
    }
}

}  // namespace norm
}  // namespace sar
