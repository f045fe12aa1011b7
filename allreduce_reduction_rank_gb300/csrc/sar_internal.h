// sar_internal.h -- launchers between the C ABI (sar_api.cu) and the kernels.
// All arguments have been validated by the caller.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <utility>

#include <cuda_runtime.h>

#include "../../include/sar.h"

namespace sar {

// Kernel launch with programmatic stream serialization: the kernel may be
// scheduled before the previous kernel in the stream has finished, and waits
// for it with pdl_wait() (sar_device.cuh) before touching memory, so the
// results are those of plain stream order.  Measured on GB300 against plain
// launches (interleaved runs): faster at every size, e.g. 2 x 16 MiB bf16
// 8.2 -> 6.1 us per call eager and 6.4 -> 6.0 us in a CUDA graph, 8 x 64 MiB
// fp16 155.8 -> 153.2 us eager.
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel_smem(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                               Args&&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, cudaStream_t s, Args&&... args) {
    return launch_kernel_smem(kernel, grid, block, 0, s, std::forward<Args>(args)...);
}

constexpr int kDevices = 64;

// Dynamic shared memory above 48 KiB is allowed explicitly, once per device and
// kernel (only a successful call is remembered).
template <class Kernel> cudaError_t allow_smem(Kernel kernel, size_t bytes, std::atomic<bool>* allowed) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (!allowed[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
        if (e != cudaSuccess) return e;
        allowed[dev].store(true, std::memory_order_release);
    }
    return cudaSuccess;
}

// What an rsag launch writes: the fused allreduce writes the reduced chunk to
// every output; the reduce-scatter step writes it to the owning rank only.
enum RsagMode { kFused = 0, kReduceScatter = 1 };

struct RankPtrs {
    const void* in[SAR_MAX_RANKS];
    void* out[SAR_MAX_RANKS];
};

// rsag reduce (fused or reduce-scatter).  `vec` selects 16-byte vectors
// (every buffer 16-byte aligned).
cudaError_t launch_rsag(RsagMode mode, sar_dtype dt, int nranks, const RankPtrs& p, size_t count,
                        size_t chunk, bool vec, cudaStream_t stream);

// Fused rsag allreduce with partial sums rounded into `acc` (fp16, bf16, or
// e4m3fn for e4m3fn inputs).
cudaError_t launch_rsag_accum(sar_dtype dt, sar_dtype acc, int nranks, const RankPtrs& p, size_t count,
                              size_t chunk, bool vec, cudaStream_t stream);

// The reduce launchers of one element type (rsag_kernels.cuh): binary32
// accumulation in either mode (instantiated in rsag_<type>.cu), and fp16 /
// bf16 / native FP8 accumulation in the fused mode (rsag_<type>_acc.cu).
template <int DT>
cudaError_t launch_rsag_wide(RsagMode mode, int nranks, const RankPtrs& p, size_t count, size_t chunk, bool vec,
                             cudaStream_t s);
template <int DT>
cudaError_t launch_rsag_narrow(sar_dtype acc, int nranks, const RankPtrs& p, size_t count, size_t chunk, bool vec,
                               cudaStream_t s);

// rsag all-gather: out[j][chunk r] = out[r][chunk r], j != r (bytes).
cudaError_t launch_all_gather(int nranks, const RankPtrs& p, size_t count, size_t esize,
                              size_t chunk, bool vec, cudaStream_t stream);

// LL pack: pkts[r] <- packets of in[r] (p.out holds the packet buffers).
cudaError_t launch_ll_pack(int nranks, const RankPtrs& p, size_t bytes, uint32_t epoch,
                           bool vec, cudaStream_t stream);

// LL poll + unpack + reduce + write-back (p.in holds the packet buffers).
cudaError_t launch_ll_unpack_reduce(sar_dtype dt, int nranks, const RankPtrs& p, size_t count,
                                    uint32_t epoch, uint64_t max_spins, int32_t* status,
                                    bool vec_out, cudaStream_t stream);

// LL send + reduce + write-back in one cooperative launch.  ctrl: optional
// device epoch counter (launches << 20); with it the k-th launch uses epoch
// (k mod (2^32 - 1)) + 1.
cudaError_t launch_ll_fused(sar_dtype dt, int nranks, const RankPtrs& data, void* const* pkts, size_t count,
                            uint32_t epoch, uint64_t* ctrl, uint64_t max_spins, int32_t* status, bool in16,
                            bool out16, cudaStream_t stream);

// LL with the write-back as a second packet round into `res`; multi_dest:
// each result packet is read once and written to all outputs.
cudaError_t launch_ll_writeback(sar_dtype dt, int nranks, const RankPtrs& data, void* const* pkts, void* res,
                                size_t count, uint32_t epoch, uint64_t* ctrl, bool multi_dest, uint64_t max_spins,
                                int32_t* status, bool in16, bool out16, cudaStream_t stream);

// Test support for the fixed scratch (not exported from the library; a test
// program links the object files): sets the last epoch used on `dev` and
// returns the array's device address there (nullptr if it was not looked up).
unsigned char* testing_fixed_scratch(int dev, bool set_epoch, uint32_t last_epoch);

// LL through distributed shared memory: one cluster of nranks CTAs per slice
// (ll_cluster.cu); nranks <= SAR_LL_CLUSTER_MAX_RANKS.
cudaError_t launch_ll_cluster(sar_dtype dt, int nranks, const RankPtrs& p, size_t count, uint64_t max_spins,
                              int32_t* status, bool in16, bool out16, cudaStream_t stream);

// LL of a small call inside one CTA, every rank's packets in its shared
// memory (ll_cta.cu); the slots take ll_cta_slot_bytes(), at most
// kLLCtaMaxSlotBytes.
constexpr size_t kLLCtaMaxSlotBytes = size_t(64) << 10;
size_t ll_cta_slot_bytes(int nranks, size_t count, sar_dtype dt);
cudaError_t launch_ll_cta(sar_dtype dt, int nranks, const RankPtrs& p, size_t count, uint64_t max_spins,
                          int32_t* status, bool in16, bool out16, cudaStream_t stream);
// The same over a grid: CTA b plays every rank for one slice of the packets
// (ll_cta.cu); any size, no scratch.
cudaError_t launch_ll_slice(sar_dtype dt, int nranks, const RankPtrs& p, size_t count, uint64_t max_spins,
                            int32_t* status, bool in16, bool out16, cudaStream_t stream);

cudaError_t launch_convert(const void* src, sar_dtype src_dt, void* dst, sar_dtype dst_dt,
                           size_t count, bool vec, cudaStream_t stream);

size_t esize_of(sar_dtype dt);

// Layer norm (layer_norm.cu).  Leading dimensions in elements; weight, bias,
// mean, rstd of the forward call and dweight, dbias of the backward call may
// be null.
struct NormArgs {
    const void* x;
    size_t ldx;
    const void* weight;
    const void* bias;
    void* y;
    size_t ldy;
    float* mean;
    float* rstd;
    size_t rows, cols;
    float eps;
};
cudaError_t launch_layer_norm(sar_dtype dt, sar_dtype wdt, const NormArgs& a, cudaStream_t stream);

struct NormGradArgs {
    const void* dy;
    size_t lddy;
    const void* x;
    size_t ldx;
    const void* weight;
    const float* mean;
    const float* rstd;
    void* dx;
    size_t lddx;
    void* dweight;
    void* dbias;
    size_t rows, cols;
    float* partial;      // layer_norm_partials(rows, cols) rows of 2 * cols sums
};
size_t layer_norm_partials(size_t rows, size_t cols);
cudaError_t launch_layer_norm_backward(sar_dtype dt, sar_dtype wdt, const NormGradArgs& a, cudaStream_t stream);

// Tokens to experts and back (experts.cu).
struct SortArgs {
    const void* ids;
    uint32_t slots;
    int experts, align;
    uint32_t capacity;
    int32_t* counts;
    int32_t* offsets;
    int32_t* position;
    int32_t* source;
};
cudaError_t launch_expert_sort(int id_bytes, const SortArgs& a, cudaStream_t stream);

struct ExpertArgs {
    const void* tok;         // tokens x cols: x of the dispatch, dout of the backward call
    size_t ldt;
    const void* rows_in;     // capacity x cols: the rows that the combine calls read
    size_t ldi;
    void* out;               // rows (dispatch), out (combine), drows (backward)
    size_t ldo;
    const int32_t* position;
    const int32_t* counts;   // null: no padding to clear
    const int32_t* offsets;
    const void* weights;     // null: every weight is 1
    void* dweights;          // null: not wanted
    int experts, topk;
    uint32_t capacity;
    size_t tokens, cols;
};
cudaError_t launch_expert_dispatch(size_t esize, const ExpertArgs& a, cudaStream_t stream);
cudaError_t launch_expert_combine(sar_dtype dt, sar_dtype wdt, const ExpertArgs& a, cudaStream_t stream);
cudaError_t launch_expert_combine_backward(sar_dtype dt, sar_dtype wdt, const ExpertArgs& a, cudaStream_t stream);


// The router (route.cu).
struct RouteArgs {
    const void* logits;
    size_t ldl;
    void* ids;               // read by the backward call
    void* weights;           // dweights of the backward call
    void* dlogits;           // backward call only
    size_t ldd;
    size_t tokens;
    int topk, experts;
    sar_softmax softmax;
};
cudaError_t launch_expert_route(sar_dtype dt, sar_dtype wdt, int id_bytes, const RouteArgs& a, cudaStream_t stream);
cudaError_t launch_expert_route_backward(sar_dtype dt, sar_dtype wdt, int id_bytes, const RouteArgs& a, cudaStream_t stream);

// The expert layer of a few tokens (expert_layer.cu).
struct LayerArgs {
    const void* x;
    size_t ldx;
    const void* ids;
    const void* weights;     // null: every weight is 1
    const void* w_in;
    const void* w_out;
    void* out;
    size_t ldo;
    int tokens, topk, experts, cols, hidden;
    bool gated;
    sar_activation activation;
    void* workspace;
};
size_t expert_layer_workspace_bytes(size_t slots, size_t cols, size_t hidden);
cudaError_t launch_expert_layer(sar_dtype dt, sar_dtype wdt, int id_bytes, const LayerArgs& a, cudaStream_t stream);

// Newton-Schulz iteration (orthogonalize.cu).
struct OrthogonalizeArgs {
    const void* g;
    size_t ldg, gstride;
    void* out;
    size_t ldo, ostride;
    size_t batch, rows, cols;
    int steps;
    float a, b, c, eps, scale;
    float grown;             // no singular value of an iterate is above
    void* workspace;
};
size_t orthogonalize_workspace_bytes(size_t batch, size_t rows, size_t cols);
cudaError_t launch_orthogonalize(sar_dtype dt, const OrthogonalizeArgs& a, cudaStream_t stream);

}  // namespace sar
