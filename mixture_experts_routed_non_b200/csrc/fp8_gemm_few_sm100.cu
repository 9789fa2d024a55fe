// Block-scaled e4m3 products for segments of a few rows, with e8m0 scales on both
// sides: decode batches and single tokens, bound by reading the weights once.
//
// Operands swapped: 128 weight rows on the MMA's M side, a chunk of up to CN = 32
// (64) rows of `a` on its N side, so that a tile's arithmetic follows the few rows
// there are (N is always CN: what lies behind the chunk's rows is never read back).  tcgen05.mma.kind::mxf8f6f4.block_scale applies the scales
// (layout in TMEM: fp8_gemm_mx_sm100.cu) and sums the unit's K in one TMEM
// accumulator; two accumulators alternate between units.  With SwiGLU a unit has
// two weight tiles (256 rows: 128 columns of h).
//
// Few units: a cluster of S CTAs shares a unit, each taking 1/S of K, so that all
// SMs pull on memory even when one token meets one matrix.  Each CTA leaves its
// partial sums in its shared memory; the CTAs then share out the tokens, and each
// adds the S partial sums of its tokens in rank order (no atomics: the result does
// not depend on timing) and writes them.
//
// Eight stages of 128 K keep 130 KB or more of weights in flight per SM.
//
// Warp roles: 0 = TMA of the weights, 1 = TMEM allocator and MMA issuer, 2 = TMA of
// the rows or gather relay, 3 idle, 4-7 = scales (one per TMEM lane quarter), 8-11 =
// epilogue, 12-13 = row gather (gathered rows only).  Every wait is bounded
// (common.cuh); one that gives up raises the CTA's abort flag, on which every role
// runs out without storing, and the error word gets MOE_DEVERR_TIMEOUT.
#include "fp8_mx.cuh"

namespace moe {
namespace {

constexpr int kFM = 128;                  // weight rows per MMA
constexpr uint32_t kFTileW = kFM * kPK;   // 16 KB
constexpr int kFGather = 64;              // gather threads
constexpr int kFMaxSplit = 8;
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
    static constexpr size_t kTableOff = (kMiscOff + 16 + 15) / 16 * 16;
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
// Cluster-scope release and acquire: shared-memory data handed to another CTA.
__device__ __forceinline__ void mbar_arrive_cluster_release(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void fence_acquire_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t cluster_addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}

struct FUnit {
    int e, nt, m0, nv;  // expert, weight tile, first sorted position, rows
};

// kS: K splits (CTAs per cluster).
template <int CN, int kMode, bool kGather>
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
    if (warp == 1) {
        tmem_alloc(smem_u32(&misc[0]), C::kTmem);
        tmem_relinquish();
    }
    if (kMode != kFp8Y16) pdl_wait();
    pdl_launch_dependents();
    load_offsets(a, off_s, kThreads);
    __syncthreads();
    if (warp == 0) {
        prefix_pieces(off_s, pre_s, E, CN, lane);
        // nothing to do when the metadata found more pairs than the arrays hold
        if (lane == 0) misc[3] = a.hdr && __ldcg(&a.hdr->abort) ? 0u : (uint32_t)pre_s[E];
    }
    tc_fence_before();
    if (S > 1) cluster_sync_all();  // the peers' barriers are initialised before any remote arrive
    else __syncthreads();
    tc_fence_after();

    const uint32_t tmem_base = misc[0];
    volatile uint32_t *abort = &misc[1];
    const bool concat = kMode == kFp8SwiGlu && a.layout == MOE_LAYOUT_CONCATENATED;
    const int n_tiles = kMode == kFp8SwiGlu ? a.N / 256 : (a.N + kFM - 1) / kFM;
    const int units = (int)misc[3] * n_tiles;  // below 2^31 (the launch sees to it)
    const int u0 = S > 1 ? (int)blockIdx.x / S : (int)blockIdx.x, du = S > 1 ? (int)gridDim.x / S : (int)gridDim.x;
    // this CTA's share of the scale blocks along K
    const int kb0 = (int)((long long)a.nk * rank / S), kb1 = (int)((long long)a.nk * (rank + 1) / S);
    // unit u: experts in order, inside one its weight tiles, inside a tile its chunks
    auto unit_of = [&](int u) {
        int lo = 0, hi = E - 1;  // the expert whose units hold u (empty experts hold none)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre_s[mid] * n_tiles <= u) lo = mid;
            else hi = mid - 1;
        }
        const int ch = pre_s[lo + 1] - pre_s[lo];
        const int rem = u - pre_s[lo] * n_tiles;
        FUnit q;
        q.e = lo;
        q.nt = ch == 1 ? rem : rem / ch;
        const int c0 = (rem - q.nt * ch) * CN;
        q.m0 = off_s[lo] + c0;
        q.nv = min(CN, off_s[lo + 1] - q.m0);
        return q;
    };
    // first weight row of tile t (0 or 1) of a unit
    auto wrow = [&](int nt, int t) {
        if (kMode != kFp8SwiGlu) return nt * kFM;
        return concat ? t * (a.N / 2) + nt * kFM : nt * 2 * kFM + t * kFM;
    };

    if (warp == 0) {
        // -------------------------------------------------- producer: weights
        const bool leader = elect_one();
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = u0; ok && u < units; u += du) {
            const FUnit q = unit_of(u);
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort));
                if (!ok) break;
                if (leader) {
                    const uint32_t fb = full_bar(stage), dst = base + stage * C::kStage;
                    mbar_arrive_expect_tx(fb, C::kStageW + (kGather ? 0u : C::kStageA));
#pragma unroll
                    for (int t = 0; t < C::kAcc; ++t)
                        tma_load_3d(dst + t * kFTileW, &a.tmap_w, fb, kb * kPK, wrow(q.nt, t), q.e);
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
        for (int u = u0; ok && u < units; u += du) {
            const FUnit q = unit_of(u);
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
        const int ha = e8m0_rows(as, nk | kb0), hw = e8m0_rows(ws, nk | kb0);
        const uint32_t sf0 = tmem_base + ((uint32_t)(32 * (warp & 3)) << 16) + C::kScale0;
        int slot = 0;
        uint32_t phase = 0;
        // a group of four blocks is loaded while the one before is handed over, a unit's row
        // numbers a unit ahead (fp8_gemm_mx_sm100.cu)
        FUnit q = {};
        int srow[kR], nrow[kR];
        size_t wi[C::kAcc];
        uint32_t ra[kR][2], rw[C::kAcc][2];
        auto load_rows = [&](int u) {
            if (u < units) q = unit_of(u);
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                const int j = 32 * i + lane;
                nrow[i] = u < units && j < q.nv ? (kGather ? __ldg(a.gather + q.m0 + j) : q.m0 + j) : -1;
            }
        };
        auto enter_unit = [&]() {  // the unit load_rows has just been called for
#pragma unroll
            for (int i = 0; i < kR; ++i) srow[i] = nrow[i] < a.rows ? nrow[i] : -1;
#pragma unroll
            for (int t = 0; t < C::kAcc; ++t) wi[t] = ((size_t)q.e * nb + wrow(q.nt, t) / kFM) * nk;
        };
        auto load_group = [&](int kb) {
            const int last = kb1 - 1 - kb;
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                ra[i][0] = 0x7F7F7F7Fu;
                ra[i][1] = 0;
                if (srow[i] >= 0) load_e8m0_x4(as, (size_t)srow[i] * nk + kb, last, ha, ra[i][0], ra[i][1]);
            }
#pragma unroll
            for (int t = 0; t < C::kAcc; ++t) load_e8m0_x4(ws, wi[t] + kb, last, hw, rw[t][0], rw[t][1]);
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
                for (int i = 0; i < kR; ++i) ca[i] = ra[i][0] | ra[i][1] << 16;
#pragma unroll
                for (int t = 0; t < C::kAcc; ++t) cw[t] = rw[t][0] | rw[t][1] << 16;
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
                tmem_st_x4(sf + 4 * C::kAcc, ca[0], ca[kR - 1], ca[kR - 1], ca[kR - 1]);
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
        for (int u = u0; u < units; u += du, ++it) {
            const FUnit q = unit_of(u);
            const uint32_t b = it & 1u;
            mbar_wait_bounded(tfull_bar(b), (it >> 1) & 1u, abort);
            // the partial sums of the unit before have been read, here and by the peers
            mbar_wait_bounded(rempty_bar, (it & 1u) ^ 1u, abort);
            __syncwarp();
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
            if (lane == 0) {
                mbar_arrive(tempty_bar(b));
                if (S == 1) mbar_arrive(rfull_bar);
            }
            if (S > 1 && lane < S) mbar_arrive_cluster_release(mapa_shared(rfull_bar, lane));
            mbar_wait_bounded(rfull_bar, it & 1u, abort);
            if (S > 1) fence_acquire_cluster();
            __syncwarp();
            const bool ok = *abort == 0;

            // Tokens rank, rank + S, ...: eight at a time, 16 threads each, eight neighbouring
            // columns per thread.
            const int c8 = (tid & 15) * 8;
            for (int j0 = rank; j0 < q.nv; j0 += 8 * S) {
                const int j = j0 + (tid >> 4) * S;
                const bool has = j < q.nv;
                const int jj = has ? j : j0;
                auto sum8 = [&](int t, int row, float (&v)[8]) {  // weight rows row .. row + 7 of tile t
                    const uint32_t at = (uint32_t)((t * CN + jj) * kFM + row) * 4u;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = 0.f;
                    for (int s = 0; s < S; ++s) {
                        float4 x, y;
                        if (S > 1) {
                            const uint32_t src = mapa_shared(red + at, (uint32_t)s);
                            x = ld_cluster_f4(src);
                            y = ld_cluster_f4(src + 16);
                        } else {
                            x = *reinterpret_cast<const float4 *>(base_ptr + C::kRedOff + at);
                            y = *reinterpret_cast<const float4 *>(base_ptr + C::kRedOff + at + 16);
                        }
                        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
                        v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
                    }
                };
                auto add_bias8 = [&](int col, float (&v)[8]) {
                    if (!a.bias) return;
                    const __nv_bfloat16 *br = a.bias + (size_t)q.e * a.N + col;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] += __bfloat162float(br[i]);
                };
                const size_t p = (size_t)q.m0 + jj;
                bool outside = false;  // a gathered row outside `a` counts as zeros
                if (kGather) {
                    const int src = __ldg(a.gather + p);
                    outside = src < 0 || src >= a.rows;
                }
                auto keep = [&](float (&v)[8]) {
                    if (kGather && outside)
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = 0.f;
                };
                if (kMode != kFp8SwiGlu) {
                    const int n = q.nt * kFM + c8;  // N is a multiple of 8: the eight are all inside or all past it
                    float v[8];
                    sum8(0, c8, v);
                    keep(v);
                    if (n < a.N) add_bias8(n, v);
                    if (kMode == kFp8Bf16) {
                        if (ok && has && n < a.N)
                            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + p * a.N + n) =
                                make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                           pack_bf16x2(v[6], v[7]));
                    } else {  // fp16 scaled by a power of two per 32 columns: four neighbouring threads
                        float m = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) m = amax_of(m, v[i]);
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                        const int ex = y_block_exp(m);
                        const float sc = exp2i(-ex);
                        if (ok && has) {
                            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + p * a.N + n) =
                                make_uint4(pack_f16x2(v[0] * sc, v[1] * sc), pack_f16x2(v[2] * sc, v[3] * sc),
                                           pack_f16x2(v[4] * sc, v[5] * sc), pack_f16x2(v[6] * sc, v[7] * sc));
                            if ((tid & 3) == 0)
                                static_cast<int8_t *>(a.out_scale)[p * (a.N / kYBlock) + n / kYBlock] = (int8_t)ex;
                        }
                    }
                } else {
                    // columns c8 .. c8 + 7 of the unit's 128 of h.  Interleaved: tile c8 / 64 holds
                    // gate and up of column c in rows 2 (c % 64), 2 (c % 64) + 1; concatenated: tile
                    // 0 the gates, tile 1 the ups
                    float g[8], up[8];
                    if (concat) {
                        sum8(0, c8, g);
                        sum8(C::kAcc - 1, c8, up);
                        keep(g);
                        keep(up);
                        add_bias8(q.nt * 128 + c8, g);
                        add_bias8(a.N / 2 + q.nt * 128 + c8, up);
                    } else {
                        float x[8], y[8];
                        const int t = c8 >> 6, row = 2 * (c8 & 63);
                        sum8(t, row, x);
                        sum8(t, row + 8, y);
                        keep(x);
                        keep(y);
                        add_bias8(q.nt * 256 + 2 * c8, x);
                        add_bias8(q.nt * 256 + 2 * c8 + 8, y);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            g[i] = x[2 * i], up[i] = x[2 * i + 1];
                            g[4 + i] = y[2 * i], up[4 + i] = y[2 * i + 1];
                        }
                    }
                    float m = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        g[i] = inf_to_nan(__fdividef(g[i], 1.0f + __expf(-g[i])) * up[i]);
                        m = amax_of(m, g[i]);
                    }
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const uint32_t e = e4m3_scale_exp(m);
                    const float is = inv_scale_of_exp(e);
                    if (ok && has) {
                        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + p * (a.N / 2) + q.nt * 128 + c8) =
                            make_uint2(pack_e4m3x4(g[0] * is, g[1] * is, g[2] * is, g[3] * is),
                                       pack_e4m3x4(g[4] * is, g[5] * is, g[6] * is, g[7] * is));
                        if ((tid & 15) == 0)
                            static_cast<uint8_t *>(a.out_scale)[p * (a.N / 256) + q.nt] = (uint8_t)e;
                    }
                }
            }
            __syncwarp();
            if (S == 1) {
                if (lane == 0) mbar_arrive(rempty_bar);
            } else if (lane < S) {
                mbar_arrive_cluster_release(mapa_shared(rempty_bar, lane));
            }
        }
    } else if (kGather && warp >= 12) {
        // -------------------------------------------------------- row gather
        // thread g: 16-byte piece (g & 7) of rows (g >> 3) + 8 i, to row * 128 +
        // ((piece ^ (row & 7)) << 4) (the 128-byte swizzle); sources as in fp8_pair.cuh
        const int g = (int)threadIdx.x - 384;
        const int piece = g & 7, r0 = g >> 3;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = u0; ok && u < units; u += du) {
            const FUnit q = unit_of(u);
            int row[CN / 8];  // -1: not copied
#pragma unroll
            for (int i = 0; i < CN / 8; ++i)
                row[i] = r0 + 8 * i < q.nv ? (int)min((long long)max(__ldg(a.gather + q.m0 + r0 + 8 * i), 0),
                                                      (long long)a.rows - 1)
                                           : -1;
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort));
                if (!ok) break;
                const uint32_t dst =
                    base + stage * C::kStage + C::kStageW + r0 * 128 + ((piece ^ (r0 & 7)) << 4);
                const uint8_t *src = a.a + min(kb * kPK + piece * 16, a.K - 16);
#pragma unroll
                for (int i = 0; i < CN / 8; ++i)
                    if (row[i] >= 0) cp_async_16(dst + i * 1024, src + (size_t)row[i] * a.K);
                cp_async_arrive_noinc(gfull_bar(stage));
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        cp_async_wait_all();
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
}

template <int CN, int kMode, bool kGather>
cudaError_t launch_one(Fp8GemmArgs &a, int num_sms, cudaStream_t s) {
    using C = FCfg<CN, kMode>;
    auto *kernel = fp8_few_kernel<CN, kMode, kGather>;
    int unused = 0;
    cudaError_t err = launch_setup_once((const void *)kernel, &unused, [&](int, int *v) -> cudaError_t {
        *v = 1;
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    });
    if (err != cudaSuccess) return err;
    {
        const uint64_t dims[3] = {(uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.E};
        const uint64_t strides[2] = {(uint64_t)a.K, (uint64_t)a.K * a.N};
        const uint32_t box[3] = {kPK, kFM, 1};
        if (!make_map_u8(&a.tmap_w, a.w, 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    if (!kGather) {
        const uint64_t dims[2] = {(uint64_t)a.K, (uint64_t)a.rows};
        const uint64_t strides[1] = {(uint64_t)a.K};
        const uint32_t box[2] = {kPK, CN};
        if (!make_map_u8(&a.tmap_a, a.a, 2, dims, strides, box)) return cudaErrorInvalidValue;
    }
    // no more chunks than P / CN and one begun per expert
    const int n_tiles = kMode == kFp8SwiGlu ? a.N / 256 : (a.N + kFM - 1) / kFM;
    const int64_t units = (a.P / CN + (a.E < a.P ? a.E : a.P)) * n_tiles;
    if (units > INT32_MAX / 2) return cudaErrorInvalidValue;  // 32-bit unit numbers in the kernel
    // Split K while the clusters still fit one to an SM each and keep two groups of four blocks
    int S = 1;
    while (S < kFMaxSplit && units * S * 2 <= num_sms && a.nk >= 8 * S) S *= 2;
    a.split = S;
    int64_t clusters = num_sms / S;
    if (clusters > units) clusters = units;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * S));
    cfg.blockDim = dim3(kGather ? 448 : 384);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (a.pdl) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (S > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = (unsigned)S;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, kernel, (const Fp8GemmArgs)a);
}

}  // namespace

cudaError_t launch_fp8_few_gemm(int mode, Fp8GemmArgs &a, int num_sms, cudaStream_t s) {
    // chunks of 32 rows where the segments hold no more than that on average
    const bool few = a.P <= 32ll * a.E;
    if (mode == kFp8SwiGlu)
        return few ? launch_one<32, kFp8SwiGlu, true>(a, num_sms, s) : launch_one<64, kFp8SwiGlu, true>(a, num_sms, s);
    if (mode == kFp8Y16)
        return few ? launch_one<32, kFp8Y16, false>(a, num_sms, s) : launch_one<64, kFp8Y16, false>(a, num_sms, s);
    if (a.gather)
        return few ? launch_one<32, kFp8Bf16, true>(a, num_sms, s) : launch_one<64, kFp8Bf16, true>(a, num_sms, s);
    return few ? launch_one<32, kFp8Bf16, false>(a, num_sms, s) : launch_one<64, kFp8Bf16, false>(a, num_sms, s);
}

}  // namespace moe
