// Block-scaled e4m3 products for segments of a few rows, with e8m0 scales on both
// sides: decode batches and single tokens, bound by reading the weights once.
//
// tcgen05.mma.kind::mxf8f6f4.block_scale applies the scales (layout in TMEM:
// fp8_gemm_mx_sm100.cu) and sums the unit's K in one TMEM accumulator; two
// accumulators alternate between units.  Units, K split and epilogue: fp8_few.cuh.
//
// The ring (up to eight stages of 128 K) keeps 131 KB of weights in flight per SM in chunks of
// 32 rows, 98 KB in chunks of 64 and 66 KB of 128.  1 x 7168 x 4096: 9.0 us, 3.3 TB/s (ramp
// and join of the split); 1024 skewed rows over 256 experts, K 512, N 2048: 32 us,
// 77 % of the rate at which the experts in use can be read.
//
// Warp roles: 0 = TMA of the weights, 1 = TMEM allocator and MMA issuer, 2 = TMA of
// the rows or gather relay, 3 idle, 4-7 = scales (one per TMEM lane quarter), 8-11 =
// epilogue, 12-13 = row gather (gathered rows only).  Every wait is bounded
// (common.cuh); one that gives up raises the CTA's abort flag, on which every role
// runs out, the cluster's output becomes NaN, and the error word gets MOE_DEVERR_TIMEOUT.
#include "fp8_few.cuh"
#include "fp8_mx.cuh"

namespace moe {
namespace {

constexpr int kFSlots = 4;                // scale slots, of four blocks each

template <int CN, int kMode>
struct FCfg {
    static constexpr int kAcc = kMode == kFp8SwiGlu ? 2 : 1;     // weight tiles per unit
    static constexpr uint32_t kStageW = kAcc * kFTileW;
    static constexpr uint32_t kStageA = CN * kPK;
    static constexpr uint32_t kStage = kStageW + kStageA;
    static constexpr uint32_t kRed = kAcc * CN * kFM * 4;        // partial sums [tile][token][weight row]
    static constexpr int kFit = (int)((200704u - kRed) / kStage);
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr uint32_t kScaleCols = 4 * kAcc + 4;         // weights' scales, then the rows'
    static constexpr uint32_t kScale0 = 2 * kAcc * CN;           // TMEM column of the first scale slot
    static constexpr uint32_t kTmemUsed = kScale0 + kFSlots * kScaleCols;
    static constexpr uint32_t kTmem = kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
    static_assert(kTmemUsed <= 512, "TMEM columns");
    static constexpr int kBars = 3 * kStages + 7 + 2 * kFSlots;
    static constexpr size_t kRedOff = (size_t)kStages * kStage;
    static constexpr size_t kBarOff = kRedOff + kRed;
    static constexpr size_t kMiscOff = kBarOff + 8 * kBars + 8;
    static constexpr size_t kFirstOff = (kMiscOff + 16 + 15) / 16 * 16;
    static constexpr size_t kTableOff = kFirstOff + kFListed * 16;
    static constexpr size_t kSmem = 1024 + kTableOff + 2 * (kMaxExperts + 1) * 4;
    static_assert(kSmem <= 232448, "shared memory of one CTA (227 KB)");
};

__device__ __forceinline__ void umma_mx(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
}
template <int CN, int kMode, bool kGather, bool kOne>
__global__ void __launch_bounds__(kGather ? 448 : 384, 1) fp8_few_kernel(const __grid_constant__ Fp8GemmArgs a) {
    using C = FCfg<CN, kMode>;
    constexpr int kThreads = kGather ? 448 : 384;
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
    auto sfull_bar = [&](int g) { return drain_bar + 8u * (3 + g); };
    auto sempty_bar = [&](int g) { return drain_bar + 8u * (3 + kFSlots + g); };
    uint32_t *misc = reinterpret_cast<uint32_t *>(base_ptr + C::kMiscOff);
    int *off_s = reinterpret_cast<int *>(base_ptr + C::kTableOff);
    int *pre_s = off_s + (kMaxExperts + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = a.E, S = a.split;
    const int rank = S > 1 ? (int)cluster_ctarank() : 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1 + (kGather ? 1 : 0));  // the producer's arrive (+ TMA bytes), the relay
            mbar_init(empty_bar(s), 1);
            mbar_init(gfull_bar(s), kFGather);
        }
        for (int g = 0; g < kFSlots; ++g) {
            mbar_init(sfull_bar(g), 4);
            mbar_init(sempty_bar(g), 1);
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
    const int units = (kOne ? ((int)a.P + CN - 1) / CN : (int)misc[3]) * n_tiles;  // below 2^31 (fp8_sizes_ok)
    const int u0 = S > 1 ? (int)blockIdx.x / S : (int)blockIdx.x, du = S > 1 ? (int)gridDim.x / S : (int)gridDim.x;
    // this CTA's share of the scale blocks along K
    const int kb0 = (int)((long long)a.nk * rank / S), kb1 = (int)((long long)a.nk * (rank + 1) / S);
    FUnits<CN, kMode, kOne> list{off_s,   pre_s,      reinterpret_cast<int4 *>(base_ptr + C::kFirstOff), 0, E, a.N,
                                 n_tiles, (int)a.P, concat};
    list.fill(units, u0, du);

    if (warp == 0) {
        // -------------------------------------------------- producer: weights
        const bool leader = elect_one();
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
                    mbar_arrive_expect_tx(fb, C::kStageW + (kGather ? 0u : C::kStageA));
#pragma unroll
                    for (int t = 0; t < C::kAcc; ++t)
                        tma_load_3d(dst + t * kFTileW, &a.tmap_w, fb, kb * kPK, list.wrow(q.nt, t), q.e);
                }
                __syncwarp();
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (!kGather && warp == 2) {
        // ----------------------------------------------------- producer: rows
        if (kMode == kFp8Y16) pdl_wait();
        const bool leader = elect_one();
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = u0, n = 0; ok && u < units; u += du, ++n) {
            const FUnit q = list.at(u, n);
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort));
                if (!ok) break;
                if (leader)
                    tma_load_2d(base + stage * C::kStage + C::kStageW, &a.tmap_a, full_bar(stage), kb * kPK, q.m0);
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
        constexpr uint32_t idesc = idesc_mx_e4m3(kFM, CN);
        int stage = 0, slot = 0;
        uint32_t phase = 0, sphase = 0, it = 0;
        bool ok = true;
        for (int u = u0; ok && u < units; u += du, ++it) {
            const uint32_t b = it & 1u, d = tmem_base + b * C::kAcc * CN;
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(tempty_bar(b), ((it >> 1) & 1u) ^ 1u, abort));
            for (int kb = kb0; ok && kb < kb1; ++kb) {
                const int k = (kb - kb0) & 3;
                if (k == 0) ok = __all_sync(0xffffffffu, mbar_wait_bounded(sfull_bar(slot), sphase, abort));
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(full_bar(stage), phase, abort)) && ok;
                if (!ok) break;
                tc_fence_after();
                const uint64_t dw = desc0 + (uint32_t)stage * (C::kStage >> 4), dx = dw + (C::kStageW >> 4);
                const uint32_t sf = tmem_base + C::kScale0 + (uint32_t)slot * C::kScaleCols;
                const uint32_t id = idesc | idesc_byte(k);
                const bool group_end = k == 3 || kb == kb1 - 1;
                if (leader) {
#pragma unroll
                    for (int t = 0; t < C::kAcc; ++t)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_mx(d + t * CN, dw + t * (kFTileW >> 4) + 2 * kk, dx + 2 * kk, id, sf + 4 * t,
                                    sf + 4 * C::kAcc, kb > kb0 || kk > 0 ? 1u : 0u);
                    umma_commit(empty_bar(stage));
                    if (kb == kb1 - 1) umma_commit(tfull_bar(b));
                    if (group_end) umma_commit(sempty_bar(slot));
                }
                __syncwarp();
                if (group_end && ++slot == kFSlots) {
                    slot = 0;
                    sphase ^= 1u;
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
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
        // ------------------------------------------------------------ scales
        if (kMode == kFp8Y16) pdl_wait();
        constexpr int kR = CN / 32;  // rows of `a` per lane
        const int nb = (a.N + 127) / 128, nk = a.nk;
        const uint8_t *as = static_cast<const uint8_t *>(a.a_scale), *ws = static_cast<const uint8_t *>(a.w_scale);
        const uint32_t sf0 = tmem_base + ((uint32_t)(32 * (warp & 3)) << 16) + C::kScale0;
        int slot = 0;
        uint32_t phase = 0;
        // a group of four blocks is loaded while the one before is handed over, a unit's row
        // numbers a unit ahead (fp8_gemm_mx_sm100.cu)
        FUnit q = {};
        int srow[kR], nrow[kR];
        size_t wi[C::kAcc];
        uint32_t ra[kR][2], rw[C::kAcc][2], shifts;
        int listed = 0;  // calls so far: the CTA's unit they are at
        auto load_rows = [&](int u) {
            if (u < units) q = list.at(u, listed++);
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                const int j = 32 * i + lane;
                nrow[i] = u < units && j < q.nv ? (kGather ? load_now(a.gather + q.m0 + j) : q.m0 + j) : -1;
            }
        };
        auto enter_unit = [&]() {  // the unit load_rows has just been called for
#pragma unroll
            for (int i = 0; i < kR; ++i) srow[i] = nrow[i] < a.rows ? nrow[i] : -1;
#pragma unroll
            for (int t = 0; t < C::kAcc; ++t) wi[t] = ((size_t)q.e * nb + list.wrow(q.nt, t) / kFM) * nk;
        };
        auto load_group = [&](int kb) {
            const int last = kb1 - 1 - kb;
            shifts = 0;
#pragma unroll
            for (int i = 0; i < kR; ++i)  // (-1: some row's scales, for accumulator columns that are dropped)
                load_e8m0_x4(as, (size_t)max(srow[i], 0) * nk + kb, last, ra[i][0], ra[i][1], shifts);
#pragma unroll
            for (int t = 0; t < C::kAcc; ++t) load_e8m0_x4(ws, wi[t] + kb, last, rw[t][0], rw[t][1], shifts);
        };
        bool ok = true;
        if (u0 < units) {
            load_rows(u0);
            enter_unit();
            load_group(kb0);
            load_rows(u0 + du);
        }
        for (int u = u0; ok && u < units; u += du) {
            for (int kb = kb0; ok && kb < kb1; kb += 4) {
                uint32_t ca[kR], cw[C::kAcc];
#pragma unroll
                for (int i = 0; i < kR; ++i) ca[i] = e8m0_word(ra[i][0], ra[i][1], shifts, kR + C::kAcc - 1 - i);
#pragma unroll
                for (int t = 0; t < C::kAcc; ++t) cw[t] = e8m0_word(rw[t][0], rw[t][1], shifts, C::kAcc - 1 - t);
                if (kb + 4 < kb1) {
                    load_group(kb + 4);
                } else if (u + du < units) {
                    enter_unit();
                    load_group(kb0);
                    load_rows(u + 2 * du);
                }
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(sempty_bar(slot), phase ^ 1u, abort));
                if (!ok) break;
                const uint32_t sf = sf0 + (uint32_t)slot * C::kScaleCols;
                tc_fence_after();
#pragma unroll
                for (int t = 0; t < C::kAcc; ++t) tmem_st_x4(sf + 4 * t, cw[t], cw[t], cw[t], cw[t]);
                // (columns past the chunk's CN rows are not read)
                tmem_st_x4(sf + 4 * C::kAcc, ca[0], ca[kR > 1 ? 1 : 0], ca[kR > 2 ? 2 : 0], ca[kR > 3 ? 3 : 0]);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sfull_bar(slot));
                if (++slot == kFSlots) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp >= 8 && warp < 12) {
        // ---------------------------------------------------------- epilogue
        const int q4 = warp & 3, tid = (int)threadIdx.x - 256;
        const uint32_t red = base + (uint32_t)C::kRedOff;
        float *red_s = reinterpret_cast<float *>(base_ptr + C::kRedOff);
        uint32_t it = 0;
        for (int u = u0, n = 0; u < units; u += du, ++n, ++it) {
            const FUnit q = list.at(u, n);
            const uint32_t b = it & 1u;
            FGone<CN> gone;
            if (kGather) gone.load(a, q, lane);
            epi_wait(tfull_bar(b), (it >> 1) & 1u, abort, S);
            // the partial sums of the unit before have been read, here and by the peers
            epi_wait(rempty_bar, (it & 1u) ^ 1u, abort, S);
            __syncwarp();
            if (kGather) gone.look(a);
            tc_fence_after();
#pragma unroll
            for (int t = 0; t < C::kAcc; ++t)
#pragma unroll
                for (int n0 = 0; n0 < CN; n0 += 32)
                    if (n0 < q.nv) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(32 * q4) << 16) + (b * C::kAcc + t) * CN + n0, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j)  // (columns past the rows: whatever is there, never read)
                            red_s[(t * CN + n0 + j) * kFM + 32 * q4 + lane] = __uint_as_float(v[j]);
                    }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(b));
            partials_ready(rfull_bar, it & 1u, S, lane, abort);
            few_output<CN, kMode, kGather>(a, q, rank, S, tid, concat, red, base_ptr + C::kRedOff, gone);
            partials_read(rempty_bar, S, lane);
        }
    } else if (kGather && warp >= 12) {
        // -------------------------------------------------------- row gather
        if constexpr (kGather)
            gather_chunk_rows<CN, kMode, kStages, C::kStage, C::kStageW>(a, list, units, u0, du, kb0, kb1,
                                                                     (int)threadIdx.x - 384, base, empty_bar,
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
    if (*abort && warp >= 8 && warp < 12) nan_units(a, list, units, u0, du, rank, S, (int)threadIdx.x - 256);
}

template <int CN, int kMode, bool kGather, bool kOne>
cudaError_t launch_one(Fp8GemmArgs &a, int num_sms, cudaStream_t s) {
    using C = FCfg<CN, kMode>;
    auto *kernel = fp8_few_kernel<CN, kMode, kGather, kOne>;
    if (!make_few_maps(a, CN, !kGather)) return cudaErrorInvalidValue;
    return launch_few(kernel, kMode, a, CN, kGather ? 448 : 384, C::kSmem, num_sms, s);
}

}  // namespace

cudaError_t launch_fp8_few_gemm(int mode, Fp8GemmArgs &a, int chunk, int num_sms, cudaStream_t s) {
    const bool c32 = chunk == 32;
    if (chunk == 128)  // one segment only
        return mode == kFp8Bf16 && !a.expert_off ? launch_one<128, kFp8Bf16, false, true>(a, num_sms, s) : cudaErrorInvalidValue;
    if (mode == kFp8SwiGlu)
        return c32 ? launch_one<32, kFp8SwiGlu, true, false>(a, num_sms, s) : launch_one<64, kFp8SwiGlu, true, false>(a, num_sms, s);
    if (mode == kFp8Y16)
        return c32 ? launch_one<32, kFp8Y16, false, false>(a, num_sms, s) : launch_one<64, kFp8Y16, false, false>(a, num_sms, s);
    if (a.gather)
        return c32 ? launch_one<32, kFp8Bf16, true, false>(a, num_sms, s) : launch_one<64, kFp8Bf16, true, false>(a, num_sms, s);
    if (a.expert_off)
        return c32 ? launch_one<32, kFp8Bf16, false, false>(a, num_sms, s) : launch_one<64, kFp8Bf16, false, false>(a, num_sms, s);
    return c32 ? launch_one<32, kFp8Bf16, false, true>(a, num_sms, s) : launch_one<64, kFp8Bf16, false, true>(a, num_sms, s);
}

}  // namespace moe
