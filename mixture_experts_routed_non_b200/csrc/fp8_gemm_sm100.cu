// Block-scaled e4m3 products grouped by expert on sm_100a (a dense product is one
// group):
//
//   out[p, n] = sum_kb sa[row(p), kb] sw[e, n/128, kb]
//               sum_{k in block kb} a[row(p), k] w[e, n, k]   (+ bias[e, n])
//
// with kb running over blocks of 128 along K, row(p) = p or gather[p], and the
// epilogues of Fp8Mode.  This file: the kernel for few rows where a scale is fp32
// (any value), and the choice among the four kernels.
//
// The tensor cores multiply the bare e4m3 codes of one block of 128 into an fp32
// accumulator (four tcgen05.mma.kind::f8f6f4 of K = 32) and the epilogue warps add
// that partial sum, times sa sw, to fp32 registers: the long sum over K is never held
// in less than fp32, and one multiply-add per element and block is all the scaling
// costs.  Two accumulator sets in TMEM let the MMAs of one block run while the
// epilogue drains the one before; what bounds a block is that hand-over (about 1000
// clocks there and back), not the memory, so the K split of fp8_few.cuh (units, split
// and output are there) counts here for more than SMs pulling on memory.
//
// Warp roles: 0 = TMA of the weights, 1 = TMEM allocator and MMA issuer, 2 = TMA of
// the rows or gather relay, 3 idle, 4-7 = epilogue (TMEM lane quarter warp%4), 8-9 =
// row gather (gathered rows only).  Every wait is bounded (common.cuh); one that gives
// up raises the CTA's abort flag, on which every role runs out, the cluster's output
// becomes NaN, and the error word gets MOE_DEVERR_TIMEOUT.
#include "fp8_few.cuh"

namespace moe {
namespace {

constexpr int CN = 32;  // rows per chunk

template <int kMode>
struct QCfg {
    static constexpr int kAcc = kMode == kFp8SwiGlu ? 2 : 1;           // weight tiles per unit
    static constexpr uint32_t kStageW = kAcc * kFTileW;
    static constexpr uint32_t kStageA = CN * kPK;
    static constexpr uint32_t kStage = kStageW + kStageA;
    static constexpr uint32_t kRed = kAcc * CN * kFM * 4;              // partial sums [tile][token][weight row]
    static constexpr int kFit = (int)((200704u - kRed) / kStage);
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr uint32_t kTmem = 2 * kAcc * CN;                   // 64 or 128 columns
    static constexpr int kBars = 3 * kStages + 7;
    static constexpr size_t kRedOff = (size_t)kStages * kStage;
    static constexpr size_t kScaleOff = kRedOff + kRed;                // [2][kAcc][CN] fp32
    static constexpr size_t kBarOff = kScaleOff + 2 * kAcc * CN * 4;
    static constexpr size_t kMiscOff = kBarOff + 8 * kBars + 8;
    static constexpr size_t kFirstOff = (kMiscOff + 16 + 15) / 16 * 16;
    static constexpr size_t kTableOff = kFirstOff + kFListed * 16;     // offsets, then chunks below each expert
    static constexpr size_t kSmem = 1024 + kTableOff + 2 * (kMaxExperts + 1) * 4;
    static_assert(kSmem <= 232448, "shared memory of one CTA (227 KB)");
};

__device__ __forceinline__ void q_epilogue_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int kMode, bool kGather, bool kOne>
__global__ void __launch_bounds__(kGather ? 320 : 256, 1) fp8_few_any_kernel(const __grid_constant__ Fp8GemmArgs a) {
    using C = QCfg<kMode>;
    constexpr int kThreads = kGather ? 320 : 256;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];

    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    const uint32_t bars = base + (uint32_t)C::kBarOff;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (kStages + s); };
    auto gfull_bar = [&](int s) { return bars + 8u * (2 * kStages + s); };
    auto tfull_bar = [&](int b) { return bars + 8u * (3 * kStages + b); };
    auto tempty_bar = [&](int b) { return bars + 8u * (3 * kStages + 2 + b); };
    const uint32_t drain_bar = bars + 8u * (3 * kStages + 4);
    const uint32_t rfull_bar = drain_bar + 8u, rempty_bar = drain_bar + 16u;
    uint32_t *misc = reinterpret_cast<uint32_t *>(base_ptr + C::kMiscOff);
    int *off_s = reinterpret_cast<int *>(base_ptr + C::kTableOff);
    int *pre_s = off_s + (kMaxExperts + 1);
    float *scale_s = reinterpret_cast<float *>(base_ptr + C::kScaleOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = a.E, S = a.split;
    const int rank = S > 1 ? (int)cluster_ctarank() : 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1 + (kGather ? 1 : 0));  // the producer's arrive (+ TMA bytes), the relay
            mbar_init(empty_bar(s), 1);
            mbar_init(gfull_bar(s), kFGather);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 4);
        }
        mbar_init(drain_bar, 1);
        mbar_init(rfull_bar, 4 * S);
        mbar_init(rempty_bar, 4 * S);
        misc[1] = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == 32) {
        tma_prefetch_desc(&a.tmap_w);
        if (!kGather) tma_prefetch_desc(&a.tmap_a);
    }
    if (kMode != kFp8Y16) pdl_wait();
    pdl_launch_dependents();
    if (!kOne) {
        load_offsets(a, off_s, kThreads);
        __syncthreads();
    }
    if (!kOne && warp == 0) {
        prefix_pieces(off_s, pre_s, E, a.P, CN, lane);
        // nothing to do when the metadata found more pairs than the arrays hold
        if (lane == 0) misc[3] = a.hdr && load_now(&a.hdr->abort) ? 0u : (uint32_t)pre_s[E];
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&misc[0]), C::kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    if (S > 1) cluster_sync_all();  // the peers' barriers are initialised before any remote arrive
    else __syncthreads();
    tc_fence_after();

    const uint32_t tmem_base = misc[0];
    volatile uint32_t *abort = &misc[1];
    const bool concat = kMode == kFp8SwiGlu && a.layout == MOE_LAYOUT_CONCATENATED;
    const int n_tiles = kMode == kFp8SwiGlu ? a.N / 256 : (a.N + kFM - 1) / kFM;
    FUnits<CN, kMode, kOne> list{off_s,   pre_s,      reinterpret_cast<int4 *>(base_ptr + C::kFirstOff), 0, E, a.N,
                                 n_tiles, (int)a.P, concat};
    const int units = (kOne ? ((int)a.P + CN - 1) / CN : (int)misc[3]) * n_tiles;  // below 2^31 (fp8_sizes_ok)
    const int u0 = S > 1 ? (int)blockIdx.x / S : (int)blockIdx.x, du = S > 1 ? (int)gridDim.x / S : (int)gridDim.x;
    list.fill(units, u0, du);
    // this CTA's share of the scale blocks along K
    const int kb0 = (int)((long long)a.nk * rank / S), kb1 = (int)((long long)a.nk * (rank + 1) / S);

    if (warp == 0 || (!kGather && warp == 2)) {
        // ------------------------------- producers: weights (warp 0), rows (warp 2)
        const bool leader = elect_one();
        if (kMode == kFp8Y16 && warp == 2) pdl_wait();
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = u0, n = 0; ok && u < units; u += du, ++n) {
            const FUnit q = list.at(u, n);
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort));
                if (!ok) break;
                if (leader) {
                    const uint32_t fb = full_bar(stage), dst = base + stage * C::kStage;
                    if (warp == 0) {
                        mbar_arrive_expect_tx(fb, C::kStageW + (kGather ? 0u : C::kStageA));
#pragma unroll
                        for (int t = 0; t < C::kAcc; ++t)
                            tma_load_3d(dst + t * kFTileW, &a.tmap_w, fb, kb * kPK, list.wrow(q.nt, t), q.e);
                    } else {
                        tma_load_2d(dst + C::kStageW, &a.tmap_a, fb, kb * kPK, q.m0);
                    }
                }
                __syncwarp();
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        // -------------------------------------------------------- MMA issuer
        const bool leader = elect_one();
        const uint64_t desc0 = smem_desc_sw128(base, 16, 1024);  // K-major, 8-row atoms 1024 B apart
        constexpr uint32_t idesc = idesc_e4m3_f32(kFM, CN);
        int stage = 0;
        uint32_t phase = 0, it = 0;
        bool ok = true;
        for (int u = u0; ok && u < units; u += du)
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const uint32_t b = it & 1u;
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(full_bar(stage), phase, abort)) &&
                     __all_sync(0xffffffffu, mbar_wait_bounded(tempty_bar(b), ((it >> 1) & 1u) ^ 1u, abort));
                if (!ok) break;
                tc_fence_after();
                const uint64_t dw = desc0 + (uint32_t)stage * (C::kStage >> 4), dx = dw + (C::kStageW >> 4);
                const uint32_t d = tmem_base + b * C::kAcc * CN;
                if (leader) {
#pragma unroll
                    for (int t = 0; t < C::kAcc; ++t)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f8(d + t * CN, dw + t * (kFTileW >> 4) + 2 * kk, dx + 2 * kk, idesc, kk > 0 ? 1u : 0u);
                    umma_commit(tfull_bar(b));
                    umma_commit(empty_bar(stage));
                }
                __syncwarp();
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        if (leader) {
            umma_commit(drain_bar);  // every MMA issued here completes before TMEM is freed
            if (!mbar_wait_timed(drain_bar, 0)) *abort = 1u;
        }
        __syncwarp();
    } else if (kGather && warp == 2) {
        // -------------------------------------------------------- gather relay
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = u0; ok && u < units; u += du)
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait_bounded(gfull_bar(stage), phase, abort)) {
                        ok = false;
                        break;
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(full_bar(stage));
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // ---------------------------------------------------------- epilogue
        if (kMode == kFp8Y16) pdl_wait();
        const int q4 = warp & 3, tid = (int)threadIdx.x - 128;
        const int nb = (a.N + 127) / 128, nk = a.nk;  // scale rows of one expert, scales per row
        const uint32_t red = base + (uint32_t)C::kRedOff;
        float *red_s = reinterpret_cast<float *>(base_ptr + C::kRedOff);
        uint32_t it = 0, uc = 0;
        // after a wait that gave up the warps run on over whatever is there and meet the
        // barriers; NaN is written at the end
        for (int u = u0, n = 0; u < units; u += du, ++n, ++uc) {
            const FUnit q = list.at(u, n);
            FGone<CN> gone;
            if (kGather) gone.load(a, q, lane);
            float acc[C::kAcc][CN];
#pragma unroll
            for (int t = 0; t < C::kAcc; ++t)
#pragma unroll
                for (int j = 0; j < CN; ++j) acc[t][j] = 0.f;
            // this thread's row scale and the tiles' weight scales, as bits, a block ahead
            int srow = -1;  // -1: past the rows, or outside `a` (few_output drops those)
            if (tid < q.nv) {
                srow = kGather ? load_now(a.gather + q.m0 + tid) : q.m0 + tid;
                if (srow >= a.rows) srow = -1;
            }
            size_t wi[C::kAcc];
            uint32_t sr[1] = {0}, wr[C::kAcc][1];
#pragma unroll
            for (int t = 0; t < C::kAcc; ++t) wi[t] = ((size_t)q.e * nb + list.wrow(q.nt, t) / kFM) * nk;
            auto load_block = [&](int kb) {
                if (srow >= 0) load_scale_bits(a.a_scale, a.a_f32, (size_t)srow * nk + kb, 0, sr);
#pragma unroll
                for (int t = 0; t < C::kAcc; ++t) load_scale_bits(a.w_scale, a.w_f32, wi[t] + kb, 0, wr[t]);
            };
            load_block(kb0);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const uint32_t b = it & 1u;
                float *sc = scale_s + b * C::kAcc * CN;
                if (tid < CN) {
                    const float s = srow >= 0 ? scale_of_bits(sr[0], a.a_f32) : 0.f;
#pragma unroll
                    for (int t = 0; t < C::kAcc; ++t) sc[t * CN + tid] = s * scale_of_bits(wr[t][0], a.w_f32);
                }
                if (kb + 1 < kb1) load_block(kb + 1);
                q_epilogue_bar();  // this block's scales are in; the other buffer's have all been read
                epi_wait(tfull_bar(b), (it >> 1) & 1u, abort, S);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int t = 0; t < C::kAcc; ++t) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(32 * q4) << 16) + (b * C::kAcc + t) * CN, v);
                    tmem_ld_wait();
                    if (t == C::kAcc - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(tempty_bar(b));
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        acc[t][j] = fmaf(__uint_as_float(v[j]), sc[t * CN + j], acc[t][j]);
                }
            }
            // the partial sums of the unit before have been read, here and by the peers
            epi_wait(rempty_bar, (uc & 1u) ^ 1u, abort, S);
            __syncwarp();
            if (kGather) gone.look(a);
#pragma unroll
            for (int t = 0; t < C::kAcc; ++t)
#pragma unroll
                for (int j = 0; j < CN; ++j) red_s[(t * CN + j) * kFM + 32 * q4 + lane] = acc[t][j];
            partials_ready(rfull_bar, uc & 1u, S, lane, abort);
            few_output<CN, kMode, kGather>(a, q, rank, S, tid, concat, red, base_ptr + C::kRedOff, gone);
            partials_read(rempty_bar, S, lane);
        }
    } else if (kGather && warp >= 8) {
        // -------------------------------------------------------- row gather
        if constexpr (kGather)
            gather_chunk_rows<CN, kMode, kStages, C::kStage, C::kStageW>(a, list, units, u0, du, kb0, kb1,
                                                                     (int)threadIdx.x - 256, base, empty_bar,
                                                                     gfull_bar, abort);
    }

    // ---------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (*abort) {
        if (threadIdx.x == 0 && a.err) atomicOr(a.err, MOE_DEVERR_TIMEOUT);
        const uint64_t w0 = globaltimer_ns();  // let copies and remote arrives already issued land
        while (globaltimer_ns() - w0 < 2000000ull) {
        }
    }
    if (S > 1) cluster_sync_all();  // no CTA leaves while a peer may read its partial sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::kTmem);
    }
    if (*abort && warp >= 4 && warp < 8) nan_units(a, list, units, u0, du, rank, S, (int)threadIdx.x - 128);
}

template <int kMode, bool kGather, bool kOne>
cudaError_t launch_one(Fp8GemmArgs &a, int num_sms, cudaStream_t s) {
    using C = QCfg<kMode>;
    auto *kernel = fp8_few_any_kernel<kMode, kGather, kOne>;
    if (!make_few_maps(a, CN, !kGather)) return cudaErrorInvalidValue;
    return launch_few(kernel, kMode, a, CN, kGather ? 320 : 256, C::kSmem, num_sms, s);
}

// Few rows, a scale in fp32.
cudaError_t launch_any_few(int mode, Fp8GemmArgs &a, int num_sms, cudaStream_t s) {
    if (mode == kFp8SwiGlu) return launch_one<kFp8SwiGlu, true, false>(a, num_sms, s);
    if (mode == kFp8Y16) return launch_one<kFp8Y16, false, false>(a, num_sms, s);
    if (a.gather) return launch_one<kFp8Bf16, true, false>(a, num_sms, s);
    return a.expert_off ? launch_one<kFp8Bf16, false, false>(a, num_sms, s) : launch_one<kFp8Bf16, false, true>(a, num_sms, s);
}

// How many clusters run at once (few_setup): the same for every few-row kernel, one CTA to an SM.
cudaError_t any_few_setup(int *fit) { return few_setup(fp8_few_any_kernel<kFp8Bf16, false, true>, 256, QCfg<kFp8Bf16>::kSmem, fit); }

// Which kernel.  Four: few rows or 256-row tiles on CTA pairs, scales by the tensor
// cores (both e8m0) or in the epilogue (any fp32).  Times below in us, in a graph.
//
// One segment: the kernel and chunk of least time by a straight line that fits what was
// measured within a tenth: a start, and per wave of units (or tiles) a time per block of
// 128 K; a split of K over 2 or 4 CTAs costs 2.2 more, over 8 3.5.
//   e8m0                       start  block   fp32 scales   start  block
//     few rows, chunks of 32     4.6  0.275                   4.0  0.385
//                         64     5.7  0.295
//                        128     8.0  0.325
//     pairs                      6.3  0.291                   5.7  0.49
//     2 (4) pairs to a tile   9.3 (10.3)  0.291              9.5 (11.0)  0.49, of their part of K
//   (one pair with e8m0: 5 % above the fit, 6.0 and 0.277.  Where others come as near, rows whose
//   pitch is no multiple of 32 bytes decide: 600 x 2992 x 1000 12.5 in chunks of 64, 15.0 in pairs.)
//   Measured, K 7168, N 4096    rows   16    48    96   128   256   384   512
//     chunks of 32                   10.0  14.2  20.0  20.0  35.6  51.2  66.3
//     chunks of 64                         12.4  16.1  16.2  22.1  38.6  38.8
//     chunks of 128                        13.2  14.4  15.5  19.6  25.8  26.0
//     pairs                                21.4  21.8  22.1  22.3  22.7  23.7
//     two pairs                                                          18.5
//   K 7168, rows 256, N 3584: chunks of 128 18.3; pairs 21.2, two 16.5, four 14.7; K 2048, rows
//     1000, N 1536: pairs 10.1, two 11.2
//   K 2048, N 1536: rows 128: 8.6, 8.9, 10.3, 10.6; 384: 9.1, 10.2, 12.2, 10.7; 768: 14.1,
//     10.5, 13.1, 10.9; 1024: 18.7, 15.4, 12.9, 11.0
//   fp32 scales, K 7168, N 4096: rows 128: 25.6 (chunks of 32), 33.3 (pairs); 256: 47.7,
//     34.1; 512: 90.9, 33.0, two pairs 24.3; K 7168, rows 256, N 3584: 46.8, 32.5, 22.8, four 18.2
// Segments whose chunks of 32 fit one to an SM however the rows fall (few rows or few
// experts): the same lines (3 experts of 128 rows, K 1024, N 1024: chunks of 32 7.4, pairs
// 9.0; fp32 scales 7.8, 10.6).  Other segments: only their average is known here.  e8m0, 128
// experts, K 768, N 2048, average rows 16 / 32 / 48 / 64 / 96: chunks of 32 38, 46, 62, 75,
// 101; chunks of 64 37, 39, 41, 54, 71; pairs 49, 50, 51, 51, 53; fp32 scales, rows 24 / 32:
// chunks of 32 60, 76, pairs 70, 70.  (Chunks of 128 only help near 64, and not where
// experts are unequal.)
struct Kernels {
    int chunk;  // rows; 0: pairs
    int pairs;  // that share a tile's K
    float start, block;
};
constexpr Kernels kE8m0Times[] = {{32, 0, 4.6f, 0.275f}, {64, 0, 5.7f, 0.295f}, {128, 0, 8.0f, 0.325f},
                                  {0, 1, 6.3f, 0.291f},  {0, 2, 9.3f, 0.291f},  {0, 4, 10.3f, 0.291f}};
constexpr Kernels kF32Times[] = {{32, 0, 4.0f, 0.385f}, {0, 1, 5.7f, 0.49f}, {0, 2, 9.5f, 0.49f}, {0, 4, 11.0f, 0.49f}};

// Units (tiles) of one segment, or the most that segments can make.
int64_t units_of(const Kernels &k, int mode, const Fp8GemmArgs &a) {
    if (k.chunk) return few_units(mode, a, k.chunk);
    return (a.expert_off ? a.P / kPM + (a.E < a.P ? a.E : a.P) : (a.P + kPM - 1) / kPM) * ((a.N + kPN - 1) / kPN);
}
float expected_us(const Kernels &k, int mode, const Fp8GemmArgs &a, int num_sms, int fit) {
    const int64_t units = units_of(k, mode, a);
    const int S = k.chunk ? few_split(units, a.nk, fit) : k.pairs, at_once = k.chunk ? num_sms / S : num_sms / 2;
    const float waves = (float)((units + at_once - 1) / at_once);
    // A few-row unit with SwiGLU has two weight tiles: twice the bytes of a block, which is what bounds
    // it with e8m0 scales; with fp32 scales the hand-over does, of both tiles at once.  (Layers of 1 to
    // 32 experts with 4 to 128 rows each, e8m0: on average 0.6 % slower than with the best kernel, 1.3 %
    // without the factor; fp32: 0.5 %, with the factor 1.3 %.)
    const float block = k.chunk && mode == kFp8SwiGlu && !a.a_f32 && !a.w_f32 ? 2.f * k.block : k.block;
    return k.start + block * waves * (float)((a.nk + S - 1) / S) + (S == 1 || !k.chunk ? 0.f : S < 8 ? 2.2f : 3.5f);
}
// Segments whose chunks of 32 fit one to an SM, and one segment: the kernel of least expected time.
bool by_time(int mode, const Fp8GemmArgs &a, int num_sms) {
    return !a.expert_off || units_of(kF32Times[0], mode, a) <= num_sms;
}

}  // namespace

Fp8Plan fp8_plan(int mode, const Fp8GemmArgs &a, int num_sms, int fit) {
    const bool e8m0 = !a.a_f32 && !a.w_f32;
    Fp8Plan p = {0, 1};
    if (mode == kFp8SwiGlu && a.P <= 16ll * a.E) {
        // (the lines are fitted on full chunks, whose SwiGLU and output take a microsecond longer: 8 experts of 4 rows,
        // H 2048, I 768: layer 28.2 us, in tiles 29.9)
        p.chunk = 32;
    } else if (by_time(mode, a, num_sms)) {
        float least = 0.f;
        auto pick = [&](const Kernels &k) {
            if ((k.chunk == 128 || k.pairs > 1) && a.expert_off) return;
            // pairs share a tile where all their clusters run at once and each keeps a group of four blocks
            if (k.pairs > 1 && (a.nk < 4 * k.pairs || units_of(k, mode, a) > ((fit >> (4 * k.pairs)) & 255))) return;
            const float us = expected_us(k, mode, a, num_sms, fit);
            if (least == 0.f || us < least) least = us, p.chunk = k.chunk, p.split = k.pairs;
        };
        if (e8m0) for (const Kernels &k : kE8m0Times) pick(k);
        else for (const Kernels &k : kF32Times) pick(k);
    } else {
        if (!e8m0) p.chunk = a.P <= 32ll * a.E ? 32 : 0;
        else p.chunk = a.P <= 16ll * a.E ? 32 : a.P <= 48ll * a.E ? 64 : 0;
    }
    if (p.chunk) p.split = few_split(few_units(mode, a, p.chunk), a.nk, fit);
    return p;
}

cudaError_t fp8_clusters(int *fit) { return any_few_setup(fit); }

cudaError_t launch_fp8_gemm(int mode, Fp8GemmArgs &a, int num_sms, cudaStream_t s) {
    if (a.P == 0 || a.N == 0) return cudaSuccess;
    int fit = 0;
    const cudaError_t err = any_few_setup(&fit);
    if (err != cudaSuccess) return err;
    const Fp8Plan p = fp8_plan(mode, a, num_sms, fit);
    a.split = p.split;
    if (!a.a_f32 && !a.w_f32)
        return p.chunk ? launch_fp8_few_gemm(mode, a, p.chunk, num_sms, s) : launch_fp8_mx_pair_gemm(mode, a, num_sms, s);
    return p.chunk ? launch_any_few(mode, a, num_sms, s) : launch_fp8_pair_gemm(mode, a, num_sms, s);
}

}  // namespace moe
