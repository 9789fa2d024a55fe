// Block-scaled e4m3 products for long segments with power-of-two (e8m0) scales on
// both sides: the computation of fp8_gemm_sm100.cu on CTA pairs (tile:
// fp8_pair.cuh) with the scales applied by the tensor cores.
//
// tcgen05.mma.kind::mxf8f6f4.block_scale multiplies each product by an e8m0 scale
// of its row of `a` and one of its weight row, per 32 values of K, and sums into
// an fp32 accumulator; a scale per 128 values is four equal ones.  The whole K of
// a tile stays in one TMEM accumulator, and nothing but the two operands and
// their scales moves per block.
//
// Scales in TMEM: row 32 c + l of a 128-row operand in lane l of column c, repeated
// in each lane quarter -- four columns for a CTA's 128 rows of `a`, eight for the
// tile's 256 weight rows, which both CTAs hold.  A 32-bit word carries the scales of
// four blocks of 128 K; the instruction descriptor names the byte to use.  Four scale
// warps per CTA, one per lane quarter, load the words of a group of four blocks ahead
// and store them once per group (a store per block kept the loop of wait, store and
// arrive as long as a block's MMAs).
//
// TMEM: the accumulator (256 columns) and four 16-column scale slots.  A second
// accumulator of this width does not fit beside them, so the epilogue first takes the whole
// accumulator into registers (64 per thread) and hands it back; conversion and
// stores run behind the next tile's MMAs.
//
// Bound by the tensor cores, and in long runs by their power: 8192 x 7168 x 4096 159
// us in bursts of four (3.0 PFLOP/s), back to back 188; 131072 gathered rows over 128
// experts, K 2048, N 1536 380 us (2.2), back to back 466.
//
// Warp roles: 0 = TMA of the weights, 1 = TMEM allocator and MMA issuer (even
// CTA), 2 = TMA of the rows or gather relay (fp8_gemm_pair_sm100.cu), 4-7 = scales, 8-23 = epilogue, 24-27 =
// row gather (gathered rows only).  Registers are moved to the epilogue warps
// (setmaxnreg: with gathered rows 4 x 88 + 3 x 48 per thread of the seven
// warpgroups, within the 7 x 72 of the launch; else 4 x 88 + 2 x 64 = 6 x 80).  Every wait
// is bounded (common.cuh).
#include "fp8_mx.cuh"

namespace moe {
namespace {

// registers per thread of the launch, of the epilogue warpgroups and of the others
__host__ __device__ constexpr int x_threads(bool gather) { return gather ? 896 : 768; }
constexpr int kXEpiRegs = 88;
__host__ __device__ constexpr int x_other_regs(bool gather) { return gather ? 48 : 64; }
static_assert(4 * kXEpiRegs + 3 * x_other_regs(true) <= 7 * 72 && 4 * kXEpiRegs + 2 * x_other_regs(false) <= 6 * 80,
              "the warpgroups' registers are no more than those of the launch");
constexpr uint32_t kXScaleCols = 16;  // TMEM columns of a scale slot: `a` at 0, weights at 8
constexpr int kXSlots = 4;            // scale slots, of four blocks each

template <int kMode>
struct XCfg {
    // 16-bit outputs pass through 32 KB of store buffers; the e4m3 rows of SwiGLU are whole
    // sectors per thread and are stored directly
    static constexpr int kStages = kMode == kFp8SwiGlu ? 6 : 5;
    static constexpr int kBars = 3 * kStages + 3 + 2 * kXSlots;
    static constexpr size_t kStoreOff = (size_t)kStages * kPStage;
    static constexpr size_t kMaxOff = kStoreOff + (kMode == kFp8SwiGlu ? 0 : kPEpiWarps * kPStore);  // [2][4][128]
    static constexpr size_t kBarOff = kMaxOff + 2 * 4 * 128 * 4;
    static constexpr size_t kMiscOff = kBarOff + 8 * kBars + 8;
    static constexpr size_t kFirstOff = (kMiscOff + 16 + 15) / 16 * 16;
    static constexpr size_t kTableOff = kFirstOff + kPListed * 16;
    static constexpr size_t kSmem = 1024 + kTableOff + 2 * (kMaxExperts + 1) * 4;
    static_assert(kSmem <= 232448, "shared memory of one CTA (227 KB)");
    static_assert(kPN + kXSlots * kXScaleCols <= kPTmem, "TMEM columns");
};

// D[tmem] (+)= (A * scales) (B * scales), e4m3 in, one e8m0 scale per 32 K of each row, K = 32.
__device__ __forceinline__ void umma_mx_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
}
// kSplit > 1 (one tile per cluster): kSplit pairs share the tile's K (pair_share).
template <int kMode, bool kGather, bool kOne, int kSplit>
__global__ void __cluster_dims__(2 * kSplit, 1, 1) __launch_bounds__(x_threads(kGather), 1)
    fp8_mx_pair_kernel(const __grid_constant__ Fp8GemmArgs a) {
    using C = XCfg<kMode>;
    constexpr int kPStages = C::kStages, kPThreads = x_threads(kGather);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    const uint32_t bars = base + (uint32_t)C::kBarOff;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (kPStages + s); };
    auto gfull_bar = [&](int s) { return bars + 8u * (2 * kPStages + s); };
    const uint32_t tfull_bar = bars + 8u * (3 * kPStages);
    const uint32_t tempty_bar = tfull_bar + 8u, drain_bar = tfull_bar + 16u;
    auto sfull_bar = [&](int g) { return drain_bar + 8u * (1 + g); };
    auto sempty_bar = [&](int g) { return drain_bar + 8u * (1 + kXSlots + g); };
    uint32_t *misc = reinterpret_cast<uint32_t *>(base_ptr + C::kMiscOff);
    int *off_s = reinterpret_cast<int *>(base_ptr + C::kTableOff);
    int *pre_s = off_s + (kMaxExperts + 1);
    float *max_s = reinterpret_cast<float *>(base_ptr + C::kMaxOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank() & 1u, even = cluster_ctarank() & ~1u;  // in the pair; the pair's even CTA
    const int pi = (int)even >> 1;                                                 // the pair
    const int E = a.E;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kPStages; ++s) {
            // even CTA: the producer's arrive (+ both CTAs' TMA bytes) and, with gathered rows, both
            // CTAs' relays
            mbar_init(full_bar(s), 1 + (kGather ? 2 : 0));
            mbar_init(empty_bar(s), 1);
            mbar_init(gfull_bar(s), kPGather);
        }
        for (int g = 0; g < kXSlots; ++g) {
            mbar_init(sfull_bar(g), 8);  // both CTAs' scale warps
            mbar_init(sempty_bar(g), 1);
        }
        mbar_init(tfull_bar, 1);
        mbar_init(tempty_bar, 2 * kPEpiWarps);
        mbar_init(drain_bar, 1);
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
        load_offsets(a, off_s, kPThreads);
        __syncthreads();
    }
    if (!kOne && warp == 0) {
        prefix_pieces(off_s, pre_s, E, a.P, kPM, lane);
        // nothing to do when the metadata found more pairs than the arrays hold (the same word in
        // both CTAs of the pair)
        if (lane == 0 && a.hdr && load_now(&a.hdr->abort)) pre_s[E] = 0;
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&misc[0]), kPTmem);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();  // barriers of both CTAs initialised before any remote arrive
    tc_fence_after();

    const uint32_t tmem_base = misc[0];
    volatile uint32_t *abort = &misc[1];
    const int nk = a.nk;
    const bool concat = kMode == kFp8SwiGlu && a.layout == MOE_LAYOUT_CONCATENATED;
    PTiles<kOne> list{off_s, pre_s, reinterpret_cast<int4 *>(base_ptr + C::kFirstOff), 0, E, a.N,
                      (a.N + kPN - 1) / kPN, (int)a.P, concat};
    const int tiles = list.count(), t0 = blockIdx.x / (2 * kSplit), dt = gridDim.x / (2 * kSplit);
    const int kb0 = kSplit == 1 ? 0 : nk * pi / kSplit, kb1 = kSplit == 1 ? nk : nk * (pi + 1) / kSplit;  // of K
    list.fill(t0, dt);

    if (warp < 4) {
        regs_dec<x_other_regs(kGather)>();
        if (warp == 0) {
            // ------------------------------------------------ producer: weights
            const bool leader = elect_one();
            const uint32_t full0 = mapa_shared(full_bar(0), even);
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_parity = 0;
            bool ok = true;
            for (int u = t0, i = 0; ok && u < tiles; u += dt, ++i) {
                const PTile t = list.at(u, i);
                const int wr = list.wrow(t.nt, (int)rank);
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort));
                    if (!ok) break;
                    if (leader) {
                        // both CTAs' TMA bytes (weights, and rows that are not gathered) land on
                        // the even CTA's barrier
                        if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), kGather ? 2 * kPHalf : 4 * kPHalf);
                        tma_load_3d_pair(base + stage * kPStage + kPHalf, &a.tmap_w, full0 + 8u * stage, kb * kPK, wr,
                                         t.e);
                    }
                    __syncwarp();
                    issued |= 1u << stage;
                    issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                    if (++stage == kPStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // the even CTA's full barriers count both CTAs' bytes: wait for every phase this
            // CTA issued before the CTA may exit
            if (rank == 0 && leader)
                for (int s = 0; s < kPStages; ++s)
                    if ((issued & (1u << s)) && !mbar_wait_timed(full_bar(s), (issued_parity >> s) & 1u)) *abort = 1u;
        } else if (!kGather && warp == 2) {
            // --------------------------------------------------- producer: rows
            if (kMode == kFp8Y16) pdl_wait();
            const bool leader = elect_one();
            const uint32_t full0 = mapa_shared(full_bar(0), even);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = t0, i = 0; ok && u < tiles; u += dt, ++i) {
                const PTile t = list.at(u, i);
                const int ar = t.m0 + 128 * (int)rank;
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort));
                    if (!ok) break;
                    if (leader)
                        tma_load_2d_pair(base + stage * kPStage, &a.tmap_a, full0 + 8u * stage, kb * kPK, ar);
                    __syncwarp();
                    if (++stage == kPStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        } else if (warp == 1 && rank == 0) {
            // ------------------------------------------------------ MMA issuer
            int stage = 0;
            uint32_t phase = 0, tphase = 0, sphase = 0;
            int slot = 0;
            bool ok = true;
            constexpr uint32_t idesc = idesc_mx_e4m3(kPM, kPN);
            const uint16_t pair_mask = (uint16_t)(0x3u << even);
            // operand descriptors: K-major, 128-byte rows, 8-row atoms 1024 B apart; stages and K
            // steps only move the start address (16-byte units, below 2^14), so the issue loop adds
            const uint64_t desc0 = smem_desc_sw128(base, 16, 1024);
            const bool leader = elect_one();
            for (int u = t0; ok && u < tiles; u += dt, tphase ^= 1u) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(tempty_bar, tphase ^ 1u, abort));
                for (int kb = kb0; ok && kb < kb1; ++kb) {
                    const int k = (kb - kb0) & 3;
                    if (k == 0) ok = __all_sync(0xffffffffu, mbar_wait_bounded(sfull_bar(slot), sphase, abort));
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(full_bar(stage), phase, abort)) && ok;
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t da = desc0 + (uint32_t)stage * (kPStage >> 4), db = da + (kPHalf >> 4);
                    const uint32_t sf = tmem_base + kPN + (uint32_t)slot * kXScaleCols;
                    const uint32_t id = idesc | idesc_byte(k);
                    const bool group_end = k == 3 || kb == kb1 - 1;
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_mx_pair(tmem_base, da + 2 * kk, db + 2 * kk, id, sf, sf + 8, kb > kb0 || kk > 0 ? 1u : 0u);
                        umma_commit_pair_mc(empty_bar(stage), pair_mask);
                        if (kb == kb1 - 1) umma_commit_pair_mc(tfull_bar, pair_mask);
                        if (group_end) umma_commit_pair_mc(sempty_bar(slot), pair_mask);
                    }
                    __syncwarp();
                    if (group_end && ++slot == kXSlots) {
                        slot = 0;
                        sphase ^= 1u;
                    }
                    if (++stage == kPStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // all pair MMAs issued here complete before TMEM is freed
            if (leader) {
                umma_commit_pair(drain_bar);
                if (!mbar_wait_timed(drain_bar, 0)) *abort = 1u;
            }
        } else if (kGather && warp == 2 && lane == 0) {
            // ------------------------------------------------------ gather relay
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = t0; ok && u < tiles; u += dt)
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait_bounded(gfull_bar(stage), phase, abort)) {
                        ok = false;
                        break;
                    }
                    fence_proxy_async_smem();
                    mbar_arrive_cluster(mapa_shared(full_bar(stage), even));
                    if (++stage == kPStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
        }
        __syncwarp();
    } else if (warp < 8) {
        regs_dec<x_other_regs(kGather)>();
        // ------------------------------------------------------------ scales
        if (kMode == kFp8Y16) pdl_wait();
        const int nb = (a.N + 127) / 128;
        const uint8_t *as = static_cast<const uint8_t *>(a.a_scale), *ws = static_cast<const uint8_t *>(a.w_scale);
        const uint32_t sf0 = tmem_base + ((uint32_t)(32 * (warp & 3)) << 16) + kPN;
        const uint32_t sfull0 = mapa_shared(sfull_bar(0), even);
        int slot = 0;
        uint32_t phase = 0;
        // The words of the next four blocks are loaded before the current four are handed over,
        // and a tile's row numbers a tile ahead: a tile's first scales would otherwise be two
        // dependent loads (thousands of clocks under load) behind the operands.
        PTile t;
        int srow[4], nrow[4];  // rows of `a`; -1: past the segment or outside `a` (never stored, or stored as zeros)
        size_t wi[2];
        uint32_t ra[4][2], rw[2][2], shifts;
        int listed = 0;  // calls so far: the cluster's tile they are at
        auto load_rows = [&](int u) {
            if (u < tiles) t = list.at(u, listed++);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = t.m0 + (int)rank * 128 + 32 * i + lane;
                nrow[i] = u < tiles && p < t.m_end ? (kGather ? load_now(a.gather + p) : p) : -1;
            }
        };
        auto enter_tile = [&]() {  // the tile load_rows has just been called for
#pragma unroll
            for (int i = 0; i < 4; ++i) srow[i] = nrow[i] < a.rows ? nrow[i] : -1;
            // (a half past the end of N has no scales: its columns are never stored)
#pragma unroll
            for (int h = 0; h < 2; ++h) wi[h] = ((size_t)t.e * nb + min(list.wrow(t.nt, h) / 128, nb - 1)) * nk;
        };
        auto load_group = [&](int kb) {
            const int last = kb1 - 1 - kb;
            shifts = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)  // (-1: some row's scales, for accumulator rows that are dropped)
                load_e8m0_x4(as, (size_t)max(srow[i], 0) * nk + kb, last, ra[i][0], ra[i][1], shifts);
#pragma unroll
            for (int h = 0; h < 2; ++h) load_e8m0_x4(ws, wi[h] + kb, last, rw[h][0], rw[h][1], shifts);
        };
        bool ok = true;
        if (t0 < tiles) {
            load_rows(t0);
            enter_tile();
            load_group(kb0);
            load_rows(t0 + dt);
        }
        for (int u = t0; ok && u < tiles; u += dt) {
            for (int kb = kb0; ok && kb < kb1; kb += 4) {
                uint32_t ca[4], cw[2];
#pragma unroll
                for (int i = 0; i < 4; ++i) ca[i] = e8m0_word(ra[i][0], ra[i][1], shifts, 5 - i);
#pragma unroll
                for (int h = 0; h < 2; ++h) cw[h] = e8m0_word(rw[h][0], rw[h][1], shifts, 1 - h);
                if (kb + 4 < kb1) {
                    load_group(kb + 4);
                } else if (u + dt < tiles) {
                    enter_tile();
                    load_group(kb0);
                    load_rows(u + 2 * dt);
                }
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(sempty_bar(slot), phase ^ 1u, abort));
                if (!ok) break;
                const uint32_t sf = sf0 + (uint32_t)slot * kXScaleCols;
                tc_fence_after();
                tmem_st_x4(sf, ca[0], ca[1], ca[2], ca[3]);
                tmem_st_x4(sf + 8, cw[0], cw[0], cw[0], cw[0]);
                tmem_st_x4(sf + 12, cw[1], cw[1], cw[1], cw[1]);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(sfull0 + 8u * slot);
                if (++slot == kXSlots) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp < 24) {
        regs_inc<kXEpiRegs>();
        // ------------------------------------------------------------ epilogue
        const int q4 = warp & 3, cq = (warp - 8) >> 2;
        const uint32_t buf = base + (uint32_t)C::kStoreOff + (uint32_t)(warp - 8) * kPStore;
        const uint32_t tempty0 = mapa_shared(tempty_bar, even);
        // the warp's two 32-column chunks of the accumulator: its own quarter, or (concatenated
        // SwiGLU) one of the gates and the matching one of the ups
        const int c0 = concat ? 32 * cq : 64 * cq, c1 = concat ? 128 + 32 * cq : 64 * cq + 32;
        const uint32_t tb = tmem_base + ((uint32_t)(32 * q4) << 16);
        uint32_t tphase = 0;
        // a wait that gives up raises the abort flag; the warp then runs on over whatever is there
        // (later waits give up at once) and meets the barriers; NaN is written at the end
        for (int u = t0, i = 0; u < tiles; u += dt, ++i, tphase ^= 1u) {
            const PTile t = list.at(u, i);
            epi_wait(tfull_bar, tphase, abort, 2 * kSplit);
            __syncwarp();
            tc_fence_after();
            uint32_t v0[32], v1[32];
            tmem_ld_32x32b_x32(tb + c0, v0);
            tmem_ld_32x32b_x32(tb + c1, v1);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty0);
            float acc[64];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                acc[j] = __uint_as_float(v0[j]);
                acc[32 + j] = __uint_as_float(v1[j]);
            }
            if (kSplit > 1 && !pair_share<kSplit>(acc, base, (int)rank, pi, cq, q4, lane)) continue;
            pair_output<kMode, kGather>(a, t, acc, (int)rank, cq, q4, lane, concat, buf, max_s + (i & 1) * 512);
        }
        if (lane == 0) bulk_wait0();  // this warp's stores are complete
    } else {
        regs_dec<x_other_regs(kGather)>();
        if constexpr (kGather)
            gather_rows<kPStages>(a, list, (int)rank, (int)threadIdx.x - 768, base, empty_bar, gfull_bar, abort, t0, dt);
    }

    if (kSplit > 1 && (warp < 8 || warp >= 24)) {
        __syncwarp();
        cluster_sync_all();  // the epilogue's, behind which the partial sums are there
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
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kPTmem);
    }
    if (*abort && warp >= 8 && warp < 24) nan_tiles<kMode>(a, list, tiles, t0, dt, (int)rank, (warp - 8) >> 2, warp & 3, lane);
}

template <int kMode, bool kGather, bool kOne, int kSplit>
cudaError_t launch_one(Fp8GemmArgs &a, int num_sms, cudaStream_t s) {
    auto *kernel = fp8_mx_pair_kernel<kMode, kGather, kOne, kSplit>;
    int unused = 0;
    cudaError_t err = launch_setup_once((const void *)kernel, &unused, [&](int, int *v) -> cudaError_t {
        *v = 1;
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)XCfg<kMode>::kSmem);
    });
    if (err != cudaSuccess) return err;
    {
        const uint64_t dims[3] = {(uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.E};
        const uint64_t strides[2] = {(uint64_t)a.K, (uint64_t)a.K * a.N};
        const uint32_t box[3] = {kPK, 128, 1};
        if (!make_map_u8(&a.tmap_w, a.w, 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    if (!kGather) {
        const uint64_t dims[2] = {(uint64_t)a.K, (uint64_t)a.rows};
        const uint64_t strides[1] = {(uint64_t)a.K};
        const uint32_t box[2] = {kPK, 128};
        if (!make_map_u8(&a.tmap_a, a.a, 2, dims, strides, box)) return cudaErrorInvalidValue;
    }
    if (kMode != kFp8SwiGlu && !make_map_out16(&a.tmap_out, a.out, (uint64_t)a.N, (uint64_t)a.P))
        return cudaErrorInvalidValue;
    const int n_tiles = (a.N + kPN - 1) / kPN;
    // one segment: its row tiles; else no more than P / 256 and one begun per expert
    const int64_t tiles = (kOne ? (a.P + kPM - 1) / kPM : a.P / kPM + (a.E < a.P ? a.E : a.P)) * n_tiles;
    // (split: one tile to a cluster)
    const int clusters = (int)(kSplit > 1 || tiles < num_sms / 2 ? tiles : num_sms / 2);
    return launch_maybe_pdl(kernel, dim3(2 * kSplit * clusters), dim3(x_threads(kGather)), XCfg<kMode>::kSmem, s, a.pdl != 0, a);
}

}  // namespace

cudaError_t launch_fp8_mx_pair_gemm(int mode, Fp8GemmArgs &a, int num_sms, cudaStream_t s) {
    if (mode == kFp8SwiGlu) return launch_one<kFp8SwiGlu, true, false, 1>(a, num_sms, s);
    if (mode == kFp8Y16) return launch_one<kFp8Y16, false, false, 1>(a, num_sms, s);
    if (a.gather) return launch_one<kFp8Bf16, true, false, 1>(a, num_sms, s);
    if (a.expert_off) return launch_one<kFp8Bf16, false, false, 1>(a, num_sms, s);
    if (a.split == 4) return launch_one<kFp8Bf16, false, true, 4>(a, num_sms, s);
    if (a.split == 2) return launch_one<kFp8Bf16, false, true, 2>(a, num_sms, s);
    return launch_one<kFp8Bf16, false, true, 1>(a, num_sms, s);
}

}  // namespace moe
