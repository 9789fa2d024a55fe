// Block-scaled e4m3 products for long segments where a scale is fp32 (any
// value): the computation of fp8_gemm_sm100.cu on CTA pairs (tile: fp8_pair.cuh).
//
// Four MMAs fill an accumulator of 256 TMEM columns with one scale block's sum;
// sixteen epilogue warps (four per TMEM lane quarter, 64 columns each) add it,
// times sa sw, to 64 fp32 registers per thread while the MMAs of the next block
// fill the other accumulator.  At the tensor cores' full rate a block takes 512
// clocks; what bounds it here is the hand-over of an accumulator, about 1200
// clocks of latency (barrier, TMEM load, arithmetic, barrier, in turn) that four
// warps per scheduler hide in part (8192 x 7168 x 4096 in bursts of four: 233 us =
// 2.1 PFLOP/s; with eight warps of 128 columns 340, with power-of-two scales, which
// need none of this, 159).
//
// Warp roles: 0 = TMA of the weights, 1 = TMEM allocator and MMA issuer (even CTA),
// 2 = TMA of the rows or gather relay, 3 = scale loader, 4-19 = epilogue, 20-23 =
// row gather (gathered rows only).  The scale loader runs up to eight blocks ahead
// and leaves sa sw per row and weight half in shared memory, four blocks per slot,
// so that no epilogue warp waits for global memory; it copies a group of row scales to
// shared memory while it hands over the one before (65536 gathered rows over 64 experts,
// K 2048, N 1536: 287 us; with two dependent loads per group instead 308).  The relay turns the gather
// threads' copies into one arrival on the MMA's barrier, after the proxy fence that
// the tensor cores' reads of them need.  Registers are moved to the epilogue warps
// (setmaxnreg: with gathered rows 4 x 104 + 2 x 32 per thread of the six
// warpgroups, the 6 x 80 of the launch; else 4 x 104 + 64 = 5 x 96).  The TMA and
// MMA warps run converged and elect the issuing lane only around the instructions
// themselves.  Every wait is bounded (common.cuh).
#include "fp8_pair.cuh"

namespace moe {
namespace {

// registers per thread of the launch and, moved, of the four epilogue warpgroups
__host__ __device__ constexpr int p_threads(bool gather) { return gather ? 768 : 640; }
__host__ __device__ constexpr int p_epi_regs(bool) { return 104; }
__host__ __device__ constexpr int p_other_regs(bool gather) { return gather ? 32 : 64; }
static_assert(4 * p_epi_regs(true) + 2 * p_other_regs(true) == 6 * 80 && 4 * p_epi_regs(false) + p_other_regs(false) == 5 * 96,
              "the warpgroups' registers are those of the launch");
constexpr int kPSlots = 2;                  // scale slots of four blocks: [4][2 halves][128 rows] fp32
constexpr uint32_t kPSlot = 4 * 2 * 128;    // floats

template <int kMode>
struct PCfg {
    // 16-bit outputs pass through 32 KB of store buffers; the e4m3 rows of SwiGLU are whole
    // sectors per thread and are stored directly
    static constexpr int kStages = kMode == kFp8SwiGlu ? 6 : 5;
    static constexpr int kBars = 3 * kStages + 5 + 2 * kPSlots;
    static constexpr size_t kStoreOff = (size_t)kStages * kPStage;
    static constexpr size_t kScaleOff = kStoreOff + (kMode == kFp8SwiGlu ? 0 : kPEpiWarps * kPStore);
    static constexpr size_t kMaxOff = kScaleOff + kPSlots * kPSlot * 4;  // SwiGlu: [4][128] row maxima
    static constexpr size_t kRawOff = kMaxOff + 2 * 4 * 128 * 4;   // [2][4][128] fp32 row scales
    static constexpr size_t kBarOff = kRawOff + 2 * 4 * 128 * 4;
    static constexpr size_t kMiscOff = kBarOff + 8 * kBars;
    static constexpr size_t kFirstOff = (kMiscOff + 16 + 15) / 16 * 16;
    static constexpr size_t kTableOff = kFirstOff + kPListed * 16;
    static constexpr size_t kSmem = 1024 + kTableOff + 2 * (kMaxExperts + 1) * 4;
    static_assert(kSmem <= 232448, "shared memory of one CTA (227 KB)");
};

__device__ __forceinline__ void umma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// kSplit > 1 (one tile per cluster): kSplit pairs share the tile's K (pair_share).
template <int kMode, bool kGather, bool kOne, int kSplit>
__global__ void __cluster_dims__(2 * kSplit, 1, 1) __launch_bounds__(p_threads(kGather), 1)
    fp8_pair_kernel(const __grid_constant__ Fp8GemmArgs a) {
    using C = PCfg<kMode>;
    constexpr int kPStages = C::kStages, kPThreads = p_threads(kGather);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    const uint32_t bars = base + (uint32_t)C::kBarOff;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (kPStages + s); };
    auto gfull_bar = [&](int s) { return bars + 8u * (2 * kPStages + s); };
    auto tfull_bar = [&](int b) { return bars + 8u * (3 * kPStages + b); };
    auto tempty_bar = [&](int b) { return bars + 8u * (3 * kPStages + 2 + b); };
    const uint32_t drain_bar = bars + 8u * (3 * kPStages + 4);
    auto sfull_bar = [&](int s) { return bars + 8u * (3 * kPStages + 5 + s); };
    auto sempty_bar = [&](int s) { return bars + 8u * (3 * kPStages + 5 + kPSlots + s); };
    float *scale_s = reinterpret_cast<float *>(base_ptr + C::kScaleOff);
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
            // even CTA: the producer's arrive (+ both CTAs' TMA bytes), and with gathered rows
            // both CTAs' relays
            mbar_init(full_bar(s), 1 + (kGather ? 2 : 0));
            mbar_init(empty_bar(s), 1);
            mbar_init(gfull_bar(s), kPGather);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 2 * kPEpiWarps);
        }
        for (int s = 0; s < kPSlots; ++s) {
            mbar_init(sfull_bar(s), 1);
            mbar_init(sempty_bar(s), kPEpiWarps);
        }
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
        regs_dec<p_other_regs(kGather)>();
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
            uint32_t phase = 0, it = 0;
            bool ok = true;
            constexpr uint32_t idesc = idesc_e4m3_f32(kPM, kPN);
            const uint16_t pair_mask = (uint16_t)(0x3u << even);
            // operand descriptors: K-major, 128-byte rows, 8-row atoms 1024 B apart; stages and K
            // steps only move the start address (16-byte units, below 2^14), so the issue loop adds
            const uint64_t desc0 = smem_desc_sw128(base, 16, 1024);
            const bool leader = elect_one();
            for (int u = t0; ok && u < tiles; u += dt) {
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const uint32_t b = it & 1u;
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(full_bar(stage), phase, abort)) &&
                         __all_sync(0xffffffffu, mbar_wait_bounded(tempty_bar(b), ((it >> 1) & 1u) ^ 1u, abort));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t da = desc0 + (uint32_t)stage * (kPStage >> 4), db = da + (kPHalf >> 4);
                    const uint32_t d = tmem_base + b * kPN;
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f8_pair(d, da + 2 * kk, db + 2 * kk, idesc, kk != 0 ? 1u : 0u);
                        umma_commit_pair_mc(tfull_bar(b), pair_mask);
                        umma_commit_pair_mc(empty_bar(stage), pair_mask);
                    }
                    __syncwarp();
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
        } else if (warp == 3) {
            // ------------------------------------------------------ scale loader
            if (kMode == kFp8Y16) pdl_wait();
            const int nb = (a.N + 127) / 128;
            const float *as32 = static_cast<const float *>(a.a_scale);
            // A group of four blocks' fp32 row scales is copied to shared memory (there are too few
            // registers to hold it) while the group before is multiplied and handed over, a tile's row
            // numbers are loaded a tile ahead, and lane 4 h + k holds the weight scale of half h, block k.
            float *raw_s = reinterpret_cast<float *>(base_ptr + C::kRawOff) + lane;  // [2][4 blocks][128 rows]
            const uint32_t raw_a = base + (uint32_t)C::kRawOff + 4u * lane;
            PTile t;
            int srow[4], nrow[4];  // rows of `a`; -1: past the segment or outside `a`, scale 0
            uint32_t wi = 0, nw = 0, buf = 0, inside = 0;
            int slot = 0, listed = 0;
            uint32_t phase = 0;
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
                wi = (uint32_t)(t.e * nb + min(list.wrow(t.nt, lane >> 2 & 1) / 128, nb - 1));
            };
            auto load_group = [&](int kb) {
                inside = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (srow[i] < 0) continue;
                    inside |= 1u << i;
                    if (a.a_f32) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (kb + k < kb1)
                                cp_async_4(raw_a + (buf * 512 + k * 128 + 32 * i) * 4u, as32 + (size_t)srow[i] * nk + kb + k);
                    } else {  // (beside fp32 scales of the weights)
                        uint32_t b[4];
                        load_scale_bits(a.a_scale, 0, (size_t)srow[i] * nk + kb, kb1 - 1 - kb, b);
#pragma unroll
                        for (int k = 0; k < 4; ++k) raw_s[buf * 512 + k * 128 + 32 * i] = scale_of_bits(b[k], 0);
                    }
                }
                cp_async_commit();
                uint32_t w[1];
                load_scale_bits(a.w_scale, a.w_f32, (size_t)wi * nk + min(kb + (lane & 3), kb1 - 1), 0, w);
                nw = w[0];
            };
            bool ok = true;
            if (t0 < tiles) {
                load_rows(t0);
                enter_tile();
                load_group(kb0);
                load_rows(t0 + dt);
            }
            for (int u = t0; ok && u < tiles; u += dt)
                for (int kb = kb0; kb < kb1; kb += 4) {
                    const float w = scale_of_bits(nw, a.w_f32);
                    const uint32_t in = inside, at = buf * 512;
                    buf ^= 1u;
                    if (kb + 4 < kb1) {
                        load_group(kb + 4);
                    } else if (u + dt < tiles) {
                        enter_tile();
                        load_group(kb0);
                        load_rows(u + 2 * dt);
                    } else {
                        cp_async_commit();
                    }
                    cp_async_wait<1>();  // (each lane reads what it copied itself)
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(sempty_bar(slot), phase ^ 1u, abort));
                    if (!ok) break;
                    float *sc = scale_s + slot * kPSlot + lane;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float w0 = __shfl_sync(0xffffffffu, w, k), w1 = __shfl_sync(0xffffffffu, w, 4 + k);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float s = raw_s[at + k * 128 + 32 * i];
                            if (!(in >> i & 1u)) s = 0.f;
                            sc[k * 256 + 32 * i] = s * w0;
                            sc[k * 256 + 128 + 32 * i] = s * w1;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sfull_bar(slot));
                    if (++slot == kPSlots) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            cp_async_wait_all();
        }
        __syncwarp();
    } else if (warp < 20) {
        regs_inc<p_epi_regs(kGather)>();
        // ------------------------------------------------------------ epilogue
        const int q4 = warp & 3, cq = (warp - 4) >> 2;
        const uint32_t buf = base + (uint32_t)C::kStoreOff + (uint32_t)(warp - 4) * kPStore;
        const uint32_t tempty0 = mapa_shared(tempty_bar(0), even), tempty1 = mapa_shared(tempty_bar(1), even);
        // the warp's two 32-column chunks of the accumulator: its own quarter, or (concatenated
        // SwiGLU) one of the gates and the matching one of the ups
        const int c0 = concat ? 32 * cq : 64 * cq, c1 = concat ? 128 + 32 * cq : 64 * cq + 32;
        const float *sc0 = scale_s + (concat ? 0 : (cq >> 1) * 128) + 32 * q4 + lane;  // chunk 0's weight half (chunk 1: concat, the ups)
        uint32_t it = 0, sphase = 0;
        int slot = 0;
        // a wait that gives up raises the abort flag; the warp then runs on over whatever is there
        // (later waits give up at once) and meets the barriers; NaN is written at the end
        for (int u = t0, i = 0; u < tiles; u += dt, ++i) {
            const PTile t = list.at(u, i);
            float acc[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = 0.f;
            for (int kb = kb0; kb < kb1; kb += 4) {
                epi_wait(sfull_bar(slot), sphase, abort, 2 * kSplit);
                __syncwarp();
                float f0[4], f1[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f0[k] = sc0[slot * kPSlot + k * 256];
                    f1[k] = concat ? sc0[slot * kPSlot + k * 256 + 128] : f0[k];
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (kb + k < kb1) {
                        const uint32_t b = it & 1u;
                        epi_wait(tfull_bar(b), (it >> 1) & 1u, abort, 2 * kSplit);
                        ++it;
                        __syncwarp();
                        tc_fence_after();
                        const uint32_t tb = tmem_base + ((uint32_t)(32 * q4) << 16) + b * kPN;
                        uint32_t v[32];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            tmem_ld_32x32b_x32(tb + (i == 0 ? c0 : c1), v);
                            tmem_ld_wait();
                            if (i == 1) {
                                // both loads have landed: the accumulator goes back to the MMA
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) {
                                    mbar_arrive_cluster(b ? tempty1 : tempty0);
                                    if (k == 0) mbar_arrive(sempty_bar(slot));  // every lane has its four scales
                                }
                            }
                            const float f = i == 0 ? f0[k] : f1[k];
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                acc[32 * i + j] = fmaf(__uint_as_float(v[j]), f, acc[32 * i + j]);
                        }
                    }
                }
                if (++slot == kPSlots) {
                    slot = 0;
                    sphase ^= 1u;
                }
            }
            if (kSplit > 1 && !pair_share<kSplit>(acc, base, (int)rank, pi, cq, q4, lane)) continue;
            pair_output<kMode, kGather>(a, t, acc, (int)rank, cq, q4, lane, concat, buf, max_s + (i & 1) * 512);
        }
        if (lane == 0) bulk_wait0();  // this warp's stores are complete
    } else {
        regs_dec<p_other_regs(kGather)>();
        if constexpr (kGather)
            gather_rows<kPStages>(a, list, (int)rank, (int)threadIdx.x - 640, base, empty_bar, gfull_bar, abort, t0, dt);
    }

    if (kSplit > 1 && (warp < 4 || warp >= 20)) {
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
    if (*abort && warp >= 4 && warp < 20) nan_tiles<kMode>(a, list, tiles, t0, dt, (int)rank, (warp - 4) >> 2, warp & 3, lane);
}

template <int kMode, bool kGather, bool kOne, int kSplit>
cudaError_t launch_one(Fp8GemmArgs &a, int num_sms, cudaStream_t s) {
    auto *kernel = fp8_pair_kernel<kMode, kGather, kOne, kSplit>;
    int unused = 0;
    cudaError_t err = launch_setup_once((const void *)kernel, &unused, [&](int, int *v) -> cudaError_t {
        *v = 1;
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PCfg<kMode>::kSmem);
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
    return launch_maybe_pdl(kernel, dim3(2 * kSplit * clusters), dim3(p_threads(kGather)), PCfg<kMode>::kSmem, s, a.pdl != 0, a);
}

}  // namespace

cudaError_t launch_fp8_pair_gemm(int mode, Fp8GemmArgs &a, int num_sms, cudaStream_t s) {
    if (mode == kFp8SwiGlu) return launch_one<kFp8SwiGlu, true, false, 1>(a, num_sms, s);
    if (mode == kFp8Y16) return launch_one<kFp8Y16, false, false, 1>(a, num_sms, s);
    if (a.gather) return launch_one<kFp8Bf16, true, false, 1>(a, num_sms, s);
    if (a.expert_off) return launch_one<kFp8Bf16, false, false, 1>(a, num_sms, s);
    if (a.split == 4) return launch_one<kFp8Bf16, false, true, 4>(a, num_sms, s);
    if (a.split == 2) return launch_one<kFp8Bf16, false, true, 2>(a, num_sms, s);
    return launch_one<kFp8Bf16, false, true, 1>(a, num_sms, s);
}

}  // namespace moe
