// route.cu -- the router: each token's best experts by their logits, the
// weights' softmax, and the logits' gradient.
//
// A warp takes a token.  Lane l holds the logits l, l + 32, ...: a row is read
// once, in whole lines.  A logit is compared as the whole number of the same order
// (route_key), so that infinities, NaN and -0 need no cases of their own.
//
// The best ones: the topk-th largest of the 32 lanes' largest, found by sorting
// those, is a lower bound of what is chosen; the few logits from there on (9 to 12
// of 256 for 8) move to a lane each and are ranked by comparing each with all.
// Taking the largest out topk times took 70 us for 65536 tokens, 8 of 256, most of
// it in 16 reductions over the warp a token; this takes 36, nearly all of it
// instructions.  The candidates grow faster than topk (9 on average for 8 of 256 normal
// logits, 21 for 16, 29 for 20, 40 for 24, 100 for 32), and where there are more than 32
// of them, one token in six at 20 and nearly all at 24, the choices are taken out one
// after another: 16 of 256 41 us, 20 63, 24 151, 32 199.
#include <type_traits>

#include "sar_device.cuh"
#include "sar_internal.h"

namespace sar {
namespace {

constexpr int kWarps = 8;
constexpr uint32_t kMasked = 0x007FFFFFu;      // the key of minus infinity

// Ascending with the value; -0 as +0, NaN above all: an addition's result is never
// -0 here, and its NaN is always 0x7FFFFFFF.
__device__ __forceinline__ uint32_t route_key(float x) {
    const int32_t u = __float_as_int(__fadd_rn(x, 0.0f));
    return static_cast<uint32_t>(u ^ (u >> 31 | static_cast<int32_t>(0x80000000u)));
}
__device__ __forceinline__ float route_value(uint32_t key) {
    return __uint_as_float(key ^ (~static_cast<uint32_t>(static_cast<int32_t>(key) >> 31) | 0x80000000u));
}

// The lanes' values, the largest first.
__device__ __forceinline__ uint32_t sort_lanes(uint32_t v, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int d = size >> 1; d > 0; d >>= 1) {
            const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, v, d);
            const bool up = ((lane & size) == 0) == ((lane & d) == 0);          // this lane keeps the larger
            v = up ? max(v, other) : min(v, other);
        }
    return v;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
    return x;
}

template <int DT, int WDT, typename Id, int V>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteArgs a) {
    pdl_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const size_t t = static_cast<size_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= a.tokens) return;
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        key[i] = e < a.experts ? route_key(load_elem<DT>(a.logits, t * a.ldl + static_cast<size_t>(e))) : 0u;
    }
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) best = max(best, key[i]);
    __shared__ uint64_t candidates[kWarps][32];
    const uint32_t top_key = __reduce_max_sync(0xFFFFFFFFu, best);
    const float top = top_key > kMasked ? route_value(top_key) : 0.0f;
    float total = 0.0f;
    if (a.softmax == SAR_SOFTMAX_ALL) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > kMasked) total = __fadd_rn(total, expf(__fsub_rn(route_value(key[i]), top)));
        total = warp_sum(total);
    }
    // Candidates: the logits from the topk-th largest of the lanes' largest on, or
    // all that are not masked where fewer lanes have one.
    const uint32_t from = max(__shfl_sync(0xFFFFFFFFu, sort_lanes(best, lane), a.topk - 1), kMasked + 1u);
    uint64_t* place = candidates[threadIdx.x >> 5];
    int count = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const bool is = key[i] >= from;
        const unsigned all = __ballot_sync(0xFFFFFFFFu, is);
        const int at = count + __popc(all & ((1u << lane) - 1u));
        if (is && at < 32) place[at] = static_cast<uint64_t>(key[i]) << 32 | ~static_cast<uint32_t>(i * 32 + lane);
        count += __popc(all);
    }
    __syncwarp();
    float mine = 0.0f;                         // of the choice that this lane holds
    int id = -1, rank = lane;
    if (count <= 32) {
        const uint64_t own = lane < count ? place[lane] : 0u;
        rank = 0;
        for (int c = 0; c < count; ++c) rank += place[c] > own ? 1 : 0;
        if (lane >= count) rank = lane;        // places that no candidate takes
        if (rank < a.topk && lane < count)
            id = static_cast<int>(~static_cast<uint32_t>(own)), mine = expf(__fsub_rn(route_value(static_cast<uint32_t>(own >> 32)), top));
    } else {                                   // many equal ones, or a large topk: one after another
        for (int j = 0; j < a.topk; ++j) {
            uint32_t local = 0;
            int at = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (key[i] > local) local = key[i], at = i;
            const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, local);
            if (most <= kMasked) break;
            const uint32_t e =
                __reduce_min_sync(0xFFFFFFFFu, local == most ? static_cast<uint32_t>(at * 32 + lane) : 0xFFFFFFFFu);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (e == static_cast<uint32_t>(i * 32 + lane)) key[i] = 0;
            if (lane == j) id = static_cast<int>(e), mine = expf(__fsub_rn(route_value(most), top));
        }
    }
    if (a.softmax == SAR_SOFTMAX_CHOSEN) total = warp_sum(mine);
    if (rank < a.topk) {
        const size_t s = t * static_cast<size_t>(a.topk) + static_cast<size_t>(rank);
        static_cast<Id*>(a.ids)[s] = id;
        store_elem<WDT>(a.weights, s, id >= 0 ? __fdiv_rn(mine, total) : 0.0f);
    }
}

template <int DT, int WDT, typename Id, int V>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(RouteArgs a) {
    pdl_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const size_t t = static_cast<size_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= a.tokens) return;
    // lane j: the j-th choice; the first of those with one id stands for all
    int id = -1;
    float dw = 0.0f;
    if (lane < a.topk) {
        const size_t s = t * static_cast<size_t>(a.topk) + static_cast<size_t>(lane);
        const Id given = static_cast<const Id*>(a.ids)[s];
        if (given >= 0 && given < static_cast<Id>(a.experts)) {
            id = static_cast<int>(given);
            dw = load_elem<WDT>(a.weights, s);
        }
    }
    bool again = false;                        // a lane below has this id
    for (int j = 0; j < a.topk; ++j) again |= __shfl_sync(0xFFFFFFFFu, id, j) == id && j < lane;
    const bool first = id >= 0 && !again;
    float given = dw;
    if (__any_sync(0xFFFFFFFFu, again && id >= 0)) {
        given = 0.0f;
        for (int j = 0; j < a.topk; ++j) {
            const int other = __shfl_sync(0xFFFFFFFFu, id, j);
            const float g = __shfl_sync(0xFFFFFFFFu, dw, j);
            if (other == id) given = __fadd_rn(given, g);
        }
    }
    if (!__any_sync(0xFFFFFFFFu, first)) {     // nothing to give a gradient to, whatever the logits
        for (int e = lane; e < a.experts; e += 32) store_elem<DT>(a.dlogits, t * a.ldd + static_cast<size_t>(e), 0.0f);
        return;
    }
    // The maximum passes over NaN; exp(NaN) makes the sum NaN, and that everything.
    float x[V];
    const float chosen = first ? load_elem<DT>(a.logits, t * a.ldl + static_cast<size_t>(id)) : -INFINITY;
    float top = chosen;
    bool nan = chosen != chosen;
    if (a.softmax == SAR_SOFTMAX_ALL) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = i * 32 + lane;
            x[i] = e < a.experts ? load_elem<DT>(a.logits, t * a.ldl + static_cast<size_t>(e)) : -INFINITY;
            top = fmaxf(top, x[i]);
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    bool empty = top == -INFINITY;
    if (empty) {                               // unless NaN are all that there is
        if (a.softmax == SAR_SOFTMAX_ALL) {
#pragma unroll
            for (int i = 0; i < V; ++i) nan |= x[i] != x[i];
        }
        empty = !__any_sync(0xFFFFFFFFu, nan);
        top = 0.0f;
    }
    const float p0 = first && !empty ? expf(__fsub_rn(chosen, top)) : 0.0f;
    float total = p0;
    if (a.softmax == SAR_SOFTMAX_ALL) {
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = expf(__fsub_rn(x[i], top));                       // 0 for minus infinity
            total = __fadd_rn(total, x[i]);
        }
    }
    total = warp_sum(total);
    const float scale = empty ? 0.0f : __fdiv_rn(1.0f, total);
    const float p = __fmul_rn(p0, scale);
    const float down = warp_sum(first ? __fmul_rn(p, given) : 0.0f);
    const float rest = -__fmul_rn(scale, down);
    const size_t row = t * a.ldd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        if (e < a.experts)
            store_elem<DT>(a.dlogits, row + static_cast<size_t>(e),
                           a.softmax == SAR_SOFTMAX_ALL ? __fmul_rn(x[i], rest) : 0.0f);
    }
    __syncwarp();                              // the chosen ones again, after the row
    if (first) store_elem<DT>(a.dlogits, row + static_cast<size_t>(id), __fmul_rn(p, __fsub_rn(given, down)));
}

template <int DT, int WDT, typename Id>
cudaError_t launch(bool backward, const RouteArgs& a, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((a.tokens + kWarps - 1) / kWarps)), block(kWarps * 32);
    const auto run = [&](auto v) {
        constexpr int V = decltype(v)::value;
        return backward ? launch_kernel(route_backward_kernel<DT, WDT, Id, V>, grid, block, s, a)
                        : launch_kernel(route_kernel<DT, WDT, Id, V>, grid, block, s, a);
    };
    if (a.experts <= 64) return run(std::integral_constant<int, 2>());
    if (a.experts <= 128) return run(std::integral_constant<int, 4>());
    if (a.experts <= 256) return run(std::integral_constant<int, 8>());
    if (a.experts <= 512) return run(std::integral_constant<int, 16>());
    return run(std::integral_constant<int, 32>());
}

template <int DT> cudaError_t launch(sar_dtype wdt, int id_bytes, bool backward, const RouteArgs& a, cudaStream_t s) {
    if (wdt == SAR_FP32)
        return id_bytes == 8 ? launch<DT, SAR_FP32, int64_t>(backward, a, s) : launch<DT, SAR_FP32, int32_t>(backward, a, s);
    return id_bytes == 8 ? launch<DT, DT, int64_t>(backward, a, s) : launch<DT, DT, int32_t>(backward, a, s);
}

cudaError_t launch(sar_dtype dt, sar_dtype wdt, int id_bytes, bool backward, const RouteArgs& a, cudaStream_t s) {
    switch (dt) {
    case SAR_BF16: return launch<SAR_BF16>(wdt, id_bytes, backward, a, s);
    case SAR_FP16: return launch<SAR_FP16>(wdt, id_bytes, backward, a, s);
    default: return launch<SAR_FP32>(wdt, id_bytes, backward, a, s);
    }
}

}  // namespace

cudaError_t launch_expert_route(sar_dtype dt, sar_dtype wdt, int id_bytes, const RouteArgs& a, cudaStream_t s) {
    return launch(dt, wdt, id_bytes, false, a, s);
}

cudaError_t launch_expert_route_backward(sar_dtype dt, sar_dtype wdt, int id_bytes, const RouteArgs& a, cudaStream_t s) {
    return launch(dt, wdt, id_bytes, true, a, s);
}

}  // namespace sar
