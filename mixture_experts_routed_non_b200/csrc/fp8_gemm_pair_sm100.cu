// Block-scaled e4m3 products for long segments: the computation of
// fp8_gemm_sm100.cu on CTA pairs, 256 rows of `a` by 256 weight rows per tile.
//
// A cluster of two CTAs owns a tile: CTA r holds rows [128 r, 128 r + 128) of
// `a` and weight rows [128 r, 128 r + 128) of each stage of 128 K (16 KB +
// 16 KB), and the even CTA issues tcgen05.mma.cta_group::2.kind::f8f6f4 (M = 256,
// N = 256, K = 32) for both, so each SM reads half the operand bytes per
// product that a tile of its own would need.  With SwiGLU the tile's 256
// weight rows are 128 gates and their 128 ups.
//
// Four MMAs fill an accumulator of 256 TMEM columns with one scale block's sum;
// eight epilogue warps (two per TMEM lane quarter, 128 columns each) add it,
// times sa sw, to 128 fp32 registers per thread while the MMAs of the next
// block fill the other accumulator.  At the tensor cores' full rate a block
// takes 512 clocks; draining 128 lanes x 256 columns and one multiply-add per
// element take about as long in TMEM reads as half of it, so the scaling hides
// behind the MMAs as long as an accumulator comes back within a block's time.
//
// Warp roles (16 warps): 0 = TMA producer, 1 = TMEM allocator and MMA issuer
// (even CTA) or gather relay (odd CTA), 2-3 idle, 4-11 = epilogue, 12-15 =
// row gather (gathered rows only).  Registers are moved to the epilogue warps
// (setmaxnreg: 56 + 200 + 200 + 56 per thread of the four warpgroups, the
// 4 x 128 of the launch).  Every wait is bounded (common.cuh).
#include "fp8.cuh"

namespace moe {
namespace {

constexpr int kPM = 256;                    // rows per tile
constexpr int kPN = 256;                    // weight rows per tile
constexpr int kPK = 128;                    // K per stage = one scale block
constexpr uint32_t kPHalf = 128 * kPK;      // 16 KB: one CTA's share of an operand stage
constexpr uint32_t kPStage = 2 * kPHalf;
constexpr int kPStages = 5;
constexpr int kPThreads = 512;
constexpr int kPGather = 128;
constexpr int kPEpiWarps = 8;
constexpr uint32_t kPTmem = 512;            // two accumulators of 256 columns
constexpr uint32_t kPStore = 32 * 128;      // per epilogue warp: 32 rows x 64 16-bit columns
constexpr int kPBars = 3 * kPStages + 5;
constexpr size_t kPStoreOff = (size_t)kPStages * kPStage;
constexpr size_t kPMaxOff = kPStoreOff + kPEpiWarps * kPStore;  // SwiGlu: [2][128] row maxima
constexpr size_t kPBarOff = kPMaxOff + 2 * 128 * 4;
constexpr size_t kPMiscOff = kPBarOff + 8 * kPBars;
constexpr size_t kPTableOff = kPMiscOff + 16;
constexpr size_t kPSmem = 1024 + kPTableOff + 2 * (kMaxExperts + 1) * 4;
static_assert(kPSmem <= 232448, "shared memory of one CTA (227 KB)");

__device__ __forceinline__ void umma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
template <int R>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
__device__ __forceinline__ void p_epilogue_bar() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

struct PTile {
    int e, nt, m0, m_end;
};

// 64 16-bit columns (32 packed pairs) of one row per lane: a warp whose 32 rows
// are all stored goes through shared memory and one TMA store (columns past N
// are clipped); otherwise each valid lane stores its row.
__device__ __forceinline__ void store64(const CUtensorMap *map, uint32_t buf, int lane, bool warp_full, bool valid,
                                        int row0, uint16_t *row, int col0, int N, const uint32_t (&v)[32]) {
    if (warp_full) {
        if (lane == 0) bulk_wait_read0();  // the buffer's previous store has been read
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c)
            st_shared_v4(buf + lane * 128 + ((c ^ (lane & 7)) << 4), v[4 * c], v[4 * c + 1], v[4 * c + 2],
                         v[4 * c + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(map, buf, col0, row0);
            bulk_commit();
        }
    } else if (valid) {
        uint4 *dst = reinterpret_cast<uint4 *>(row + col0);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (col0 + 8 * c < N) dst[c] = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    }
}

template <int kMode, bool kGather>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPThreads, 1)
    fp8_pair_kernel(const __grid_constant__ Fp8GemmArgs a) {
    extern __shared__ uint8_t smem_raw[];
    // uniform for both CTAs of the pair: they return together
    if (a.hdr && *(volatile const uint32_t *)&a.hdr->abort) return;

    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    const uint32_t bars = base + (uint32_t)kPBarOff;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (kPStages + s); };
    auto gfull_bar = [&](int s) { return bars + 8u * (2 * kPStages + s); };
    auto tfull_bar = [&](int b) { return bars + 8u * (3 * kPStages + b); };
    auto tempty_bar = [&](int b) { return bars + 8u * (3 * kPStages + 2 + b); };
    const uint32_t drain_bar = bars + 8u * (3 * kPStages + 4);
    uint32_t *misc = reinterpret_cast<uint32_t *>(base_ptr + kPMiscOff);
    int *off_s = reinterpret_cast<int *>(base_ptr + kPTableOff);
    int *pre_s = off_s + (kMaxExperts + 1);
    float *max_s = reinterpret_cast<float *>(base_ptr + kPMaxOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int E = a.E;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kPStages; ++s) {
            // even CTA: the producer's arrive (+ both CTAs' TMA bytes); gathered rows add the
            // even CTA's gather threads and the odd CTA's relay
            mbar_init(full_bar(s), 1 + (kGather ? 1 + kPGather : 0));
            mbar_init(empty_bar(s), 1);
            mbar_init(gfull_bar(s), kPGather);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 2 * kPEpiWarps);
        }
        mbar_init(drain_bar, 1);
        misc[1] = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == 32) {
        tma_prefetch_desc(&a.tmap_w);
        if (!kGather) tma_prefetch_desc(&a.tmap_a);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&misc[0]), kPTmem);
        tmem_relinquish_pair();
    }
    // segment offsets, held inside [0, P] whatever the caller's table says
    if (a.expert_off) {
        for (int i = threadIdx.x; i <= E; i += kPThreads)
            off_s[i] = (int)min(max((long long)__ldg(a.expert_off + i), 0ll), (long long)a.P);
    } else if (threadIdx.x < 2) {
        off_s[threadIdx.x] = threadIdx.x ? (int)a.P : 0;
    }
    __syncthreads();
    if (warp == 0) {  // pre_s[e] = row tiles of the experts below e
        int sum = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < E ? (max(off_s[e + 1] - off_s[e], 0) + kPM - 1) / kPM : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            if (e < E) pre_s[e] = sum + incl - n;
            sum += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) pre_s[E] = sum;
    }
    tc_fence_before();
    cluster_sync_all();  // barriers of both CTAs initialised before any remote arrive
    tc_fence_after();

    const uint32_t tmem_base = misc[0];
    volatile uint32_t *abort = &misc[1];
    const int nk = a.nk;
    const bool concat = kMode == kFp8SwiGlu && a.layout == MOE_LAYOUT_CONCATENATED;
    const int n_tiles = (a.N + kPN - 1) / kPN;
    const long long tiles = (long long)pre_s[E] * n_tiles;
    const long long t0 = blockIdx.x >> 1, dt = gridDim.x >> 1;
    auto tile_of = [&](long long u) {
        PTile t;
        const int mt = (int)(u / n_tiles);
        t.nt = (int)(u - (long long)mt * n_tiles);
        int lo = 0, hi = E - 1;  // largest e with pre_s[e] <= mt
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre_s[mid] <= mt) lo = mid;
            else hi = mid - 1;
        }
        t.e = lo;
        t.m0 = off_s[lo] + (mt - pre_s[lo]) * kPM;
        t.m_end = off_s[lo + 1];
        return t;
    };
    // first weight row of half h (accumulator columns 128 h ..) of a tile
    auto wrow = [&](int nt, int h) { return concat ? h * (a.N / 2) + nt * 128 : nt * kPN + h * 128; };

    if (warp < 4) {
        regs_dec<56>();
        if (warp == 0 && lane == 0) {
            // -------------------------------------------------------- producer
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_parity = 0;
            bool ok = true;
            for (long long u = t0; ok && u < tiles; u += dt) {
                const PTile t = tile_of(u);
                const int wr = wrow(t.nt, (int)rank), ar = t.m0 + 128 * (int)rank;
                for (int kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort)) {
                        ok = false;
                        break;
                    }
                    // both CTAs' TMA bytes land on the even CTA's barrier
                    if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), kGather ? 2 * kPHalf : 4 * kPHalf);
                    const uint32_t fb = mapa_shared(full_bar(stage), 0), dst = base + stage * kPStage;
                    tma_load_3d_pair(dst + kPHalf, &a.tmap_w, fb, kb * kPK, wr, t.e);
                    if (!kGather) tma_load_2d_pair(dst, &a.tmap_a, fb, kb * kPK, ar);
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
            if (rank == 0)
                for (int s = 0; s < kPStages; ++s)
                    if ((issued & (1u << s)) && !mbar_wait_timed(full_bar(s), (issued_parity >> s) & 1u)) *abort = 1u;
        } else if (warp == 1 && rank == 0 && lane == 0) {
            // ------------------------------------------------------ MMA issuer
            int stage = 0;
            uint32_t phase = 0, it = 0;
            bool ok = true;
            constexpr uint32_t idesc = idesc_e4m3_f32(kPM, kPN);
            for (long long u = t0; ok && u < tiles; u += dt) {
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const uint32_t b = it & 1u;
                    if (!mbar_wait_bounded(tempty_bar(b), ((it >> 1) & 1u) ^ 1u, abort) ||
                        !mbar_wait_bounded(full_bar(stage), phase, abort)) {
                        ok = false;
                        break;
                    }
                    if (kGather) fence_proxy_async_smem();
                    tc_fence_after();
                    const uint32_t sa = base + stage * kPStage, sb = sa + kPHalf;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)  // K-major, 128-byte rows, 8-row atoms 1024 B apart
                        umma_f8_pair(tmem_base + b * kPN, smem_desc_sw128(sa + kk * 32, 16, 1024),
                                     smem_desc_sw128(sb + kk * 32, 16, 1024), idesc, kk != 0 ? 1u : 0u);
                    umma_commit_pair_mc(empty_bar(stage), 0x3);
                    umma_commit_pair_mc(tfull_bar(b), 0x3);
                    if (++stage == kPStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // all pair MMAs issued here complete before TMEM is freed
            umma_commit_pair(drain_bar);
            if (!mbar_wait_timed(drain_bar, 0)) *abort = 1u;
        } else if (kGather && warp == 1 && rank == 1 && lane == 0) {
            // ------------------------------------------- relay (odd CTA, gathered rows)
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (long long u = t0; ok && u < tiles; u += dt)
                for (int kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait_bounded(gfull_bar(stage), phase, abort)) {
                        ok = false;
                        break;
                    }
                    fence_proxy_async_smem();
                    mbar_arrive_cluster(mapa_shared(full_bar(stage), 0));
                    if (++stage == kPStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
        }
        __syncwarp();
    } else if (warp < 12) {
        regs_inc<200>();
        // ------------------------------------------------------------ epilogue
        const int q4 = warp & 3, half = (warp - 4) >> 2;
        const int r = 32 * q4 + lane;  // row inside this CTA's 128
        const uint32_t buf = base + (uint32_t)kPStoreOff + (uint32_t)(warp - 4) * kPStore;
        const uint32_t tempty0 = mapa_shared(tempty_bar(0), 0), tempty1 = mapa_shared(tempty_bar(1), 0);
        const int nb = (a.N + 127) / 128;
        // the warp's four 32-column chunks of the accumulator: its own half, or (concatenated
        // SwiGLU) two of the gates and the matching two of the ups
        const int c0 = concat ? 2 * half : 4 * half, c2 = concat ? 4 + 2 * half : 4 * half + 2;
        uint32_t it = 0;
        bool ok = true;  // after a wait that gave up: no more waits, but the named barriers are met
        for (long long u = t0; u < tiles; u += dt) {
            const PTile t = tile_of(u);
            const int row0 = t.m0 + (int)rank * 128 + q4 * 32;
            const int p = row0 + lane;
            const bool valid = p < t.m_end;
            long long srow = -1;
            if (valid) {
                srow = kGather ? (long long)__ldg(a.gather + p) : (long long)p;
                if (srow >= a.rows) srow = -1;
            }
            const int h0 = concat ? 0 : half, h2 = concat ? 1 : half;  // the chunks' weight halves
            // (a half past the end of N has no scales: its columns are never stored)
            const int b0 = min(wrow(t.nt, h0) / 128, nb - 1), b2 = min(wrow(t.nt, h2) / 128, nb - 1);
            const size_t wi0 = ((size_t)t.e * nb + b0) * nk, wi2 = ((size_t)t.e * nb + b2) * nk;
            float s_a = 0.f;
            if (srow >= 0) s_a = load_scale(a.a_scale, a.a_f32, (size_t)srow * nk);
            float s_w0 = load_scale(a.w_scale, a.w_f32, wi0), s_w2 = concat ? load_scale(a.w_scale, a.w_f32, wi2) : s_w0;
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.f;
            for (int kb = 0; kb < nk; ++kb, ++it) {
                const uint32_t b = it & 1u;
                const float f0 = s_a * s_w0, f2 = s_a * s_w2;
                if (kb + 1 < nk) {
                    if (srow >= 0) s_a = load_scale(a.a_scale, a.a_f32, (size_t)srow * nk + kb + 1);
                    s_w0 = load_scale(a.w_scale, a.w_f32, wi0 + kb + 1);
                    s_w2 = concat ? load_scale(a.w_scale, a.w_f32, wi2 + kb + 1) : s_w0;
                }
                if (ok) {
                    bool w = true;
                    if (lane == 0) w = mbar_wait_bounded(tfull_bar(b), (it >> 1) & 1u, abort);
                    ok = __shfl_sync(0xffffffffu, w, 0);
                }
                if (!ok) continue;
                tc_fence_after();
                const uint32_t tb = tmem_base + ((uint32_t)(32 * q4) << 16) + b * kPN;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(tb + ((i < 2 ? c0 : c2) + (i & 1)) * 32, v);
                    tmem_ld_wait();
                    if (i == 3) {
                        // the block's last load has landed: the accumulator goes back to the MMA
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(b ? tempty1 : tempty0);
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        acc[32 * i + j] = fmaf(__uint_as_float(v[j]), i < 2 ? f0 : f2, acc[32 * i + j]);
                }
            }
            const bool warp_full = ok && row0 + 31 < t.m_end;
            const bool store = ok && valid;
            if (kMode != kFp8SwiGlu) {
                const int col = t.nt * kPN + half * 128;
                uint16_t *orow = static_cast<uint16_t *>(a.out) + (size_t)(valid ? p : 0) * a.N;
                if (a.bias) {
                    const __nv_bfloat16 *br = a.bias + (size_t)t.e * a.N + col;
#pragma unroll
                    for (int j = 0; j < 128; ++j)
                        if (col + j < a.N) acc[j] += __bfloat162float(br[j]);
                }
                uint32_t exps = 0;
                if (kMode == kFp8Y16) {  // fp16 scaled by a power of two per 32 columns
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float m = 0.f;
#pragma unroll
                        for (int j = 0; j < 32; ++j) m = amax_of(m, acc[32 * i + j]);
                        const int ex = y_block_exp(m);
                        const float sc = exp2i(-ex);
                        exps |= (uint32_t)(uint8_t)(int8_t)ex << (8 * i);
#pragma unroll
                        for (int j = 0; j < 32; ++j) acc[32 * i + j] *= sc;
                    }
                    if (store && col < a.N)  // N is a multiple of 128: the four exponents are one aligned word
                        *reinterpret_cast<uint32_t *>(static_cast<int8_t *>(a.out_scale) + (size_t)p * (a.N / kYBlock) +
                                                      col / kYBlock) = exps;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = kMode == kFp8Y16 ? pack_f16x2(acc[64 * i + 2 * j], acc[64 * i + 2 * j + 1])
                                                : pack_bf16x2(acc[64 * i + 2 * j], acc[64 * i + 2 * j + 1]);
                    if (col + 64 * i < a.N)
                        store64(&a.tmap_out, buf, lane, warp_full, store, row0, orow, col + 64 * i, a.N, v);
                }
            } else {
                // h = silu(gate) up: 64 columns per thread, with the other half's 64 one scale block
                const int hc = t.nt * 128 + half * 64;  // first h column of this thread
                if (a.bias) {
                    const __nv_bfloat16 *br = a.bias + (size_t)t.e * a.N;
#pragma unroll
                    for (int j = 0; j < 128; ++j) {
                        const int col = concat ? (j < 64 ? hc + j : a.N / 2 + hc + j - 64) : 2 * hc + j;
                        acc[j] += __bfloat162float(br[col]);
                    }
                }
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < 64; ++j) {
                    // interleaved: columns 2j, 2j+1; the value goes to acc[j], whose own column
                    // has been used by then (j <= 2j)
                    const float g = concat ? acc[j] : acc[2 * j], up = concat ? acc[64 + j] : acc[2 * j + 1];
                    const float h = inf_to_nan(__fdividef(g, 1.0f + __expf(-g)) * up);
                    acc[j] = h;
                    m = amax_of(m, h);
                }
                max_s[half * 128 + r] = m;
                p_epilogue_bar();
                m = fmaxf(m, max_s[(half ^ 1) * 128 + r]);
                const uint32_t e = e4m3_scale_exp(m);
                const float is = inv_scale_of_exp(e);
                if (store) {
                    uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.out) + (size_t)p * (a.N / 2) + hc);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int j = 16 * i + 4 * k;
                            v[k] = pack_e4m3x4(acc[j] * is, acc[j + 1] * is, acc[j + 2] * is, acc[j + 3] * is);
                        }
                        o[i] = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                    if (half == 0) static_cast<uint8_t *>(a.out_scale)[(size_t)p * (a.N / 256) + t.nt] = (uint8_t)e;
                }
                p_epilogue_bar();  // max_s has been read
            }
        }
        if (lane == 0) bulk_wait0();  // this warp's stores are complete
    } else {
        regs_dec<56>();
        if (kGather) {
            // --------------------------------------------------- row gather
            // thread g: 16-byte piece (g & 7) of rows (g >> 3) + 16 i, stored at
            // row * 128 + ((piece ^ (row & 7)) << 4) (the 128-byte swizzle)
            const int g = (int)threadIdx.x - 384;
            const int piece = g & 7, r0 = g >> 3;
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (long long u = t0; ok && u < tiles; u += dt) {
                const PTile t = tile_of(u);
                int row[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int p = t.m0 + (int)rank * 128 + r0 + 16 * i;
                    row[i] = p < t.m_end ? __ldg(a.gather + p) : -2;
                    if (row[i] >= a.rows || row[i] == -1) row[i] = -1;
                }
                for (int kb = 0; kb < nk; ++kb) {
                    bool w = true;
                    if (lane == 0) w = mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort);
                    w = __shfl_sync(0xffffffffu, w, 0);
                    if (!w) {
                        ok = false;
                        break;
                    }
                    const uint32_t sx = base + stage * kPStage;
                    const int k0 = kb * kPK + piece * 16;
                    const bool in = k0 < a.K;  // K is a multiple of 16
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rr = r0 + 16 * i;
                        // rows past the segment's end feed only accumulator rows that are never
                        // stored; a row outside `a` and the K past the end are zeros
                        const bool rd = in && row[i] >= 0;
                        if (row[i] != -2)
                            cp_async_16_zfill(sx + rr * 128 + ((piece ^ (rr & 7)) << 4),
                                              rd ? a.a + (size_t)row[i] * a.K + k0 : a.a, rd ? 16u : 0u);
                    }
                    cp_async_arrive_noinc(rank == 0 ? full_bar(stage) : gfull_bar(stage));
                    if (++stage == kPStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            cp_async_wait_all();
        }
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
}

template <int kMode, bool kGather>
cudaError_t launch_one(Fp8GemmArgs &a, int num_sms, cudaStream_t s) {
    auto *kernel = fp8_pair_kernel<kMode, kGather>;
    int unused = 0;
    cudaError_t err = launch_setup_once((const void *)kernel, &unused, [&](int, int *v) -> cudaError_t {
        *v = 1;
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPSmem);
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
    if (kMode != kFp8SwiGlu && !make_map_16(&a.tmap_out, a.out, (uint64_t)a.N, (uint64_t)a.P, 64, 32))
        return cudaErrorInvalidValue;
    const int n_tiles = (a.N + kPN - 1) / kPN;
    // no more row tiles than P / 256 and one begun per expert
    const int64_t tiles = (a.P / kPM + (a.E < a.P ? a.E : a.P)) * n_tiles;
    const int clusters = (int)(tiles < num_sms / 2 ? tiles : num_sms / 2);
    kernel<<<2 * clusters, kPThreads, kPSmem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_pair_gemm(int mode, Fp8GemmArgs &a, int num_sms, cudaStream_t s) {
    if (mode == kFp8SwiGlu) return launch_one<kFp8SwiGlu, true>(a, num_sms, s);
    if (mode == kFp8Y16) return launch_one<kFp8Y16, false>(a, num_sms, s);
    return a.gather ? launch_one<kFp8Bf16, true>(a, num_sms, s) : launch_one<kFp8Bf16, false>(a, num_sms, s);
}

}  // namespace moe
