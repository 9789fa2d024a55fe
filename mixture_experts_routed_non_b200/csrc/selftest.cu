// Self-test of the failure path every pipeline wait of the GEMM kernels
// takes: a bounded mbarrier wait that nothing will ever complete must give up
// after its limit, record MOE_DEVERR_TIMEOUT in the workspace's error word and
// let the kernel return normally, leaving the context usable.  No fault, trap
// or endless loop is involved.
//
// And of what the block-scaled products make of it where CTAs of a cluster share a
// unit's (tile's) K: the hand-over functions that their epilogues use, with partial sums
// of constants, and accumulators that one CTA (one pair) is never given.
#include <string.h>

#include "fp8_few.cuh"

namespace moe {
namespace {

__global__ void wait_timeout_selftest_kernel(WsHeader *hdr, unsigned long long timeout_ns) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ uint32_t abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bar), 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        // nothing arrives on the barrier: its first phase never completes
        const bool ok = mbar_wait_bounded(smem_u32(&bar), 0, &abort_flag, timeout_ns);
        if (!ok && abort_flag) atomicOr(&hdr->err, MOE_DEVERR_TIMEOUT);
    }
}

// Units of 32 rows x 128 columns, two CTAs to a unit: out = 1 + 2.  lose: CTA 1 never gets
// its accumulators from unit 1 on and goes on with something else.
constexpr int kUnits = 3;
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(128)
    few_handover_selftest_kernel(const __grid_constant__ Fp8GemmArgs a, int lose, unsigned long long timeout_ns) {
    __shared__ __align__(16) float red_s[32 * kFM];
    __shared__ __align__(8) uint64_t bars[3];
    __shared__ uint32_t abort_flag;
    const int rank = (int)cluster_ctarank(), tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t tfull_bar = smem_u32(bars), rfull_bar = tfull_bar + 8u, rempty_bar = tfull_bar + 16u;
    if (tid == 0) {
        mbar_init(tfull_bar, 1);
        mbar_init(rfull_bar, 4 * 2);
        mbar_init(rempty_bar, 4 * 2);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    cluster_sync_all();
    volatile uint32_t *abort = &abort_flag;
    const FUnits<32, kFp8Bf16, true> list = {nullptr, nullptr, nullptr, 0, 1, a.N, 1, (int)a.P, false};
    for (int u = 0; u < kUnits; ++u) {
        const FUnit q = list.at(u, u);
        const FGone<32> gone = {};
        if (tid == 0 && !(lose && rank == 1 && u >= 1)) mbar_arrive(tfull_bar);
        epi_wait(tfull_bar, u & 1u, abort, 2, timeout_ns);
        epi_wait(rempty_bar, (u & 1u) ^ 1u, abort, 2, timeout_ns);
        __syncwarp();
        for (int j = 0; j < 32; ++j)
            red_s[j * kFM + 32 * warp + lane] = lose && rank == 1 && u >= 1 ? 7.f : 1.f + (float)rank;
        partials_ready(rfull_bar, u & 1u, 2, lane, abort, timeout_ns);
        few_output<32, kFp8Bf16, false>(a, q, rank, 2, tid, false, smem_u32(red_s),
                                        reinterpret_cast<const uint8_t *>(red_s), gone);
        partials_read(rempty_bar, 2, lane);
    }
    __syncthreads();
    if (*abort && tid == 0) atomicOr(a.err, MOE_DEVERR_TIMEOUT);
    cluster_sync_all();
    if (*abort) nan_units(a, list, kUnits, 0, 1, rank, 2, tid);
}

// One tile of 256 x 256, two pairs to it: out = 1 + 2.  lose: the second pair never gets its
// accumulator.
constexpr uint32_t kShareRing = 4 * 32768u;
__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(512)
    pair_share_selftest_kernel(const __grid_constant__ Fp8GemmArgs a, int lose, unsigned long long timeout_ns) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    __shared__ __align__(8) uint64_t bar;
    __shared__ uint32_t abort_flag;
    const int rank = (int)cluster_ctarank() & 1, pi = (int)cluster_ctarank() >> 1;
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31, q4 = warp & 3, cq = warp >> 2;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bar), 1);
        abort_flag = 0;
        fence_barrier_init();
        if (!(lose && pi == 1)) mbar_arrive(smem_u32(&bar));
    }
    __syncthreads();
    cluster_sync_all();
    const PTiles<true> list = {nullptr, nullptr, nullptr, 0, 1, a.N, 1, (int)a.P, false};
    epi_wait(smem_u32(&bar), 0, &abort_flag, 4, timeout_ns);
    __syncwarp();
    float acc[64];
    for (int j = 0; j < 64; ++j) acc[j] = lose && pi == 1 ? 7.f : 1.f + (float)pi;  // unfinished: something else
    if (pair_share<2>(acc, ring, rank, pi, cq, q4, lane)) {
        pair_output<kFp8Bf16, false>(a, list.at(0, 0), acc, rank, cq, q4, lane, false, ring + kShareRing + warp * kPStore,
                                     nullptr);
        if (lane == 0) bulk_wait0();
    }
    __syncthreads();
    if (*(volatile uint32_t *)&abort_flag && threadIdx.x == 0) atomicOr(a.err, MOE_DEVERR_TIMEOUT);
    cluster_sync_all();
    if (*(volatile uint32_t *)&abort_flag) nan_tiles<kFp8Bf16>(a, list, 1, 0, 1, rank, cq, q4, lane);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" MOE_API int moe_nonexpand_selftest_wait_timeout(void *ws, size_t ws_bytes, uint32_t timeout_us,
                                                          moe_stream_t stream) {
    if (!ws || ws_bytes < sizeof(WsHeader) || (reinterpret_cast<uintptr_t>(ws) % 256) != 0) return MOE_ERR_WS;
    if (timeout_us < 1 || timeout_us > 2000000) return MOE_ERR_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    WsHeader *hdr = static_cast<WsHeader *>(ws);
    if (cudaMemsetAsync(&hdr->err, 0, sizeof(hdr->err), s) != cudaSuccess) return MOE_ERR_CUDA;
    wait_timeout_selftest_kernel<<<1, 32, 0, s>>>(hdr, (unsigned long long)timeout_us * 1000ull);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" MOE_API int moe_fp8_selftest_wait_timeout(int32_t pairs, int32_t lose, void *out, uint32_t *err_word,
                                                     uint32_t timeout_us, moe_stream_t stream) {
    if (!out || !ptr_aligned(out, 16) || !err_word || !ptr_aligned(err_word, 4)) return MOE_ERR_ARG;
    if (timeout_us < 1 || timeout_us > 2000000) return MOE_ERR_ARG;
    int sms = 0;
    const int st = current_device_sms(&sms);
    if (st) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const unsigned long long ns = (unsigned long long)timeout_us * 1000ull;
    Fp8GemmArgs a;
    memset(&a, 0, sizeof a);
    a.out = out;
    a.err = err_word;
    a.E = 1;
    if (!pairs) {
        a.P = 32 * kUnits;
        a.N = kFM;
        few_handover_selftest_kernel<<<2, 128, 0, s>>>(a, lose, ns);
    } else {
        constexpr uint32_t smem = 1024 + kShareRing + kPEpiWarps * kPStore;
        a.P = kPM;
        a.N = kPN;
        if (!make_map_out16(&a.tmap_out, out, (uint64_t)a.N, (uint64_t)a.P)) return MOE_ERR_CUDA;
        if (cudaFuncSetAttribute(pair_share_selftest_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
            cudaSuccess)
            return MOE_ERR_CUDA;
        pair_share_selftest_kernel<<<4, 512, smem, s>>>(a, lose, ns);
    }
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
