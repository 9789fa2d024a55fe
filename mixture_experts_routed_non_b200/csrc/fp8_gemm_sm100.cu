// Block-scaled e4m3 products grouped by expert on sm_100a (a dense product is
// one group):
//
//   out[p, n] = sum_kb sa[row(p), kb] sw[e, n/128, kb]
//               sum_{k in block kb} a[row(p), k] w[e, n, k]   (+ bias[e, n])
//
// with kb running over blocks of 128 along K, row(p) = p or gather[p], and the
// epilogues of Fp8Mode.  The scales are any fp32 (or e8m0), so the tensor cores
// multiply the bare e4m3 codes of one block of 128 into an fp32 accumulator
// (four tcgen05.mma.kind::f8f6f4 of K = 32) and the epilogue warps add that
// partial sum, times sa sw, to fp32 registers: the long sum over K is never held
// in less than fp32, and one fused multiply-add per element and block is all
// the scaling costs.
//
// Tile: 128 weight rows on the MMA's M side, a chunk of up to CN rows of `a` on
// its N side (CN = 32 for few rows, else 128; 64 with SwiGLU, whose two weight
// tiles of a unit -- gate and up -- need two accumulators).  A chunk's MMA N is
// its row count rounded up to 16.  Two accumulator sets in TMEM let the MMAs of
// one K block run while the epilogue drains the previous one.
//
// Warp roles (one CTA per SM, units (chunk, weight tile) dealt round-robin):
// warp 0 = TMA producer, warp 1 = TMEM allocator and MMA issuer, warps 2-5 =
// epilogue (TMEM lane quarter warp%4), warps 6-7 (gathered rows) = cp.async
// gather straight into the 128-byte swizzle.  Every wait is bounded
// (common.cuh); on a timeout the CTA raises its abort flag, records
// MOE_DEVERR_TIMEOUT, drains and returns.
#include "fp8.cuh"

namespace moe {
namespace {

constexpr int kQM = 128;                   // weight rows per MMA (M)
constexpr int kQK = 128;                   // K per stage = one scale block = one 128-byte swizzle atom
constexpr uint32_t kQTileW = kQM * kQK;    // 16 KB
constexpr int kQGatherWarps = 2;

template <int CN, int kMode>
struct QCfg {
    static constexpr int kAcc = kMode == kFp8SwiGlu ? 2 : 1;           // weight tiles per unit
    static constexpr uint32_t kStageW = kAcc * kQTileW;
    static constexpr uint32_t kStageA = CN * kQK;
    static constexpr uint32_t kStage = kStageW + kStageA;
    static constexpr int kStages = (int)(196608u / kStage) > 10 ? 10 : (int)(196608u / kStage);
    static constexpr uint32_t kTmemUsed = 2 * kAcc * CN;
    static constexpr uint32_t kTmem = kTmemUsed < 64 ? 64 : kTmemUsed;  // a power of two
    static constexpr int kBars = 2 * kStages + 5;
    static constexpr size_t kScaleOff = (size_t)kStages * kStage;       // [2][kAcc][CN] fp32
    static constexpr size_t kMaxOff = kScaleOff + 2 * kAcc * CN * 4;    // [4][CN] fp32 (SwiGlu)
    static constexpr size_t kBarOff = kMaxOff + (kMode == kFp8SwiGlu ? 4 * CN * 4 : 0);
    static constexpr size_t kMiscOff = kBarOff + 8 * kBars;
    static constexpr size_t kTableOff = kMiscOff + 16;                  // offsets, then chunk prefix
    static constexpr size_t kSmem = 1024 + kTableOff + 2 * (kMaxExperts + 1) * 4;
    static_assert(kSmem <= 232448, "shared memory of one CTA (227 KB)");
    static_assert(kTmem <= 512 && (kTmem & (kTmem - 1)) == 0, "TMEM columns");
};

__device__ __forceinline__ void q_epilogue_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

struct QUnit {
    int e, nt, m0, nv;  // expert, weight tile, first sorted position, rows
};

template <int CN, int kMode, bool kGather>
__global__ void __launch_bounds__(kGather ? 256 : 192, 1) fp8_gemm_kernel(const __grid_constant__ Fp8GemmArgs a) {
    using C = QCfg<CN, kMode>;
    constexpr int kThreads = kGather ? 256 : 192;
    extern __shared__ uint8_t smem_raw[];
    pdl_wait();  // (its dependents start when it has finished)
    if (a.hdr && *(volatile const uint32_t *)&a.hdr->abort) return;

    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    const uint32_t bars = base + (uint32_t)C::kBarOff;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (C::kStages + s); };
    auto tfull_bar = [&](int b) { return bars + 8u * (2 * C::kStages + b); };
    auto tempty_bar = [&](int b) { return bars + 8u * (2 * C::kStages + 2 + b); };
    const uint32_t drain_bar = bars + 8u * (2 * C::kStages + 4);
    uint32_t *misc = reinterpret_cast<uint32_t *>(base_ptr + C::kMiscOff);
    int *off_s = reinterpret_cast<int *>(base_ptr + C::kTableOff);
    int *pre_s = off_s + (kMaxExperts + 1);
    float *scale_s = reinterpret_cast<float *>(base_ptr + C::kScaleOff);
    float *max_s = reinterpret_cast<float *>(base_ptr + C::kMaxOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = a.E;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full_bar(s), 1 + (kGather ? 32 * kQGatherWarps : 0));
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 4);
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
        tmem_alloc(smem_u32(&misc[0]), C::kTmem);
        tmem_relinquish();
    }
    // segment offsets, held inside [0, P] whatever the caller's table says
    if (a.expert_off) {
        for (int i = threadIdx.x; i <= E; i += kThreads)
            off_s[i] = (int)min(max((long long)__ldg(a.expert_off + i), 0ll), (long long)a.P);
    } else if (threadIdx.x < 2) {
        off_s[threadIdx.x] = threadIdx.x ? (int)a.P : 0;
    }
    __syncthreads();
    if (warp == 0) {  // pre_s[e] = chunks of the experts below e
        int sum = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < E ? (max(off_s[e + 1] - off_s[e], 0) + CN - 1) / CN : 0;
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
    __syncthreads();
    tc_fence_after();

    const uint32_t tmem_base = misc[0];
    volatile uint32_t *abort = &misc[1];
    const int nk = a.nk;
    const bool concat = kMode == kFp8SwiGlu && a.layout == MOE_LAYOUT_CONCATENATED;
    const int n_tiles = kMode == kFp8SwiGlu ? a.N / 256 : (a.N + kQM - 1) / kQM;
    const long long units = (long long)pre_s[E] * n_tiles;
    // unit u: experts in order, inside one its weight tiles, inside a tile its chunks
    auto unit_of = [&](long long u) {
        int lo = 0, hi = E - 1;  // the expert whose units hold u (empty experts hold none)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((long long)pre_s[mid] * n_tiles <= u) lo = mid;
            else hi = mid - 1;
        }
        const int ch = pre_s[lo + 1] - pre_s[lo];
        const int rem = (int)(u - (long long)pre_s[lo] * n_tiles);
        QUnit q;
        q.e = lo;
        q.nt = rem / ch;
        const int c0 = (rem - q.nt * ch) * CN;
        q.m0 = off_s[lo] + c0;
        q.nv = min(CN, off_s[lo + 1] - q.m0);
        return q;
    };
    // first weight row of tile t (0 or 1) of a unit
    auto wrow = [&](int nt, int t) {
        if (kMode != kFp8SwiGlu) return nt * kQM;
        return concat ? t * (a.N / 2) + nt * kQM : nt * 2 * kQM + t * kQM;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (long long u = blockIdx.x; ok && u < units; u += gridDim.x) {
                const QUnit q = unit_of(u);
                for (int kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = full_bar(stage), sw = base + stage * C::kStage;
                    mbar_arrive_expect_tx(fb, C::kStageW + (kGather ? 0u : C::kStageA));
#pragma unroll
                    for (int t = 0; t < C::kAcc; ++t)
                        tma_load_3d(sw + t * kQTileW, &a.tmap_w, fb, kb * kQK, wrow(q.nt, t), q.e);
                    if (!kGather) tma_load_2d(sw + C::kStageW, &a.tmap_a, fb, kb * kQK, q.m0);
                    if (++stage == C::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, it = 0;
            bool ok = true;
            for (long long u = blockIdx.x; ok && u < units; u += gridDim.x) {
                const QUnit q = unit_of(u);
                const uint32_t idesc = idesc_e4m3_f32(kQM, (q.nv + 15) & ~15);
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const uint32_t b = it & 1u;
                    if (!mbar_wait_bounded(tempty_bar(b), ((it >> 1) & 1u) ^ 1u, abort) ||
                        !mbar_wait_bounded(full_bar(stage), phase, abort)) {
                        ok = false;
                        break;
                    }
                    if (kGather) fence_proxy_async_smem();
                    tc_fence_after();
                    const uint32_t sw = base + stage * C::kStage, sx = sw + C::kStageW;
#pragma unroll
                    for (int t = 0; t < C::kAcc; ++t)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)  // K-major, 128-byte rows, 8-row atoms 1024 B apart
                            umma_f8(tmem_base + (b * C::kAcc + t) * CN,
                                    smem_desc_sw128(sw + t * kQTileW + kk * 32, 16, 1024),
                                    smem_desc_sw128(sx + kk * 32, 16, 1024), idesc, kk != 0 ? 1u : 0u);
                    umma_commit(empty_bar(stage));
                    umma_commit(tfull_bar(b));
                    if (++stage == C::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            umma_commit(drain_bar);  // every MMA issued here completes before TMEM is freed
            if (!mbar_wait_timed(drain_bar, 0)) *abort = 1u;
        }
        __syncwarp();
    } else if (warp < 6) {
        // ------------------------------------------------------------ epilogue
        const int q4 = warp & 3;
        const int r = 32 * q4 + lane;             // weight row inside the tile
        const int tid = (int)threadIdx.x - 64;    // 0..127: the chunk row whose scale this thread loads
        const int nb = (a.N + kQM - 1) / kQM;     // scale rows of one expert
        uint32_t it = 0;
        // after a wait that gave up, the warp keeps meeting the others at the named barriers
        // but waits for nothing more: all four leave together
        bool ok = true;
        for (long long u = blockIdx.x; u < units; u += gridDim.x) {
            const QUnit q = unit_of(u);
            float acc[C::kAcc][CN];
#pragma unroll
            for (int t = 0; t < C::kAcc; ++t)
#pragma unroll
                for (int j = 0; j < CN; ++j) acc[t][j] = 0.f;
            // this thread's row scale and the tile's weight scales, one block ahead
            long long srow = -1;
            if (tid < q.nv) {
                srow = kGather ? (long long)__ldg(a.gather + q.m0 + tid) : (long long)q.m0 + tid;
                if (srow >= a.rows) srow = -1;
            }
            size_t wsi[C::kAcc];
#pragma unroll
            for (int t = 0; t < C::kAcc; ++t) wsi[t] = ((size_t)q.e * nb + wrow(q.nt, t) / kQM) * nk;
            float s_cur = 0.f, w_cur[C::kAcc];
            if (srow >= 0) s_cur = load_scale(a.a_scale, a.a_f32, (size_t)srow * nk);
#pragma unroll
            for (int t = 0; t < C::kAcc; ++t) w_cur[t] = load_scale(a.w_scale, a.w_f32, wsi[t]);
            for (int kb = 0; kb < nk; ++kb, ++it) {
                const uint32_t b = it & 1u;
                float *sc = scale_s + b * C::kAcc * CN;
                if (tid < CN) {
#pragma unroll
                    for (int t = 0; t < C::kAcc; ++t) sc[t * CN + tid] = s_cur * w_cur[t];
                }
                if (kb + 1 < nk) {
                    if (srow >= 0) s_cur = load_scale(a.a_scale, a.a_f32, (size_t)srow * nk + kb + 1);
#pragma unroll
                    for (int t = 0; t < C::kAcc; ++t) w_cur[t] = load_scale(a.w_scale, a.w_f32, wsi[t] + kb + 1);
                }
                q_epilogue_bar();  // this block's scales are in; the other buffer's have all been read
                if (ok) {
                    bool w = true;
                    if (lane == 0) w = mbar_wait_bounded(tfull_bar(b), (it >> 1) & 1u, abort);
                    ok = __shfl_sync(0xffffffffu, w, 0);
                }
                if (!ok) continue;
                tc_fence_after();
#pragma unroll
                for (int t = 0; t < C::kAcc; ++t)
#pragma unroll
                    for (int n0 = 0; n0 < CN; n0 += 32) {
                        if (n0 < q.nv) {
                            uint32_t v[32];
                            tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(32 * q4) << 16) + (b * C::kAcc + t) * CN + n0, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                acc[t][n0 + j] = fmaf(__uint_as_float(v[j]), sc[t * CN + n0 + j], acc[t][n0 + j]);
                        }
                    }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(tempty_bar(b));
            }
            if (kMode == kFp8Bf16) {
                const int n = q.nt * kQM + r;
                if (ok && n < a.N) {
                    const float bias = a.bias ? __bfloat162float(a.bias[(size_t)q.e * a.N + n]) : 0.f;
                    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.out) + (size_t)q.m0 * a.N + n;
#pragma unroll
                    for (int j = 0; j < CN; ++j)
                        if (j < q.nv) o[(size_t)j * a.N] = __float2bfloat16_rn(acc[0][j] + bias);
                }
            } else if (kMode == kFp8Y16) {
                // a warp's lanes hold one 32-column block of each token (N is a multiple of 128)
                const int n = q.nt * kQM + r;
                const float bias = a.bias ? __bfloat162float(a.bias[(size_t)q.e * a.N + n]) : 0.f;
                uint16_t *o = static_cast<uint16_t *>(a.out) + (size_t)q.m0 * a.N + n;
                int8_t *os = static_cast<int8_t *>(a.out_scale) + (size_t)q.m0 * (a.N / kYBlock) + n / kYBlock;
#pragma unroll
                for (int j = 0; j < CN; ++j) {
                    if (j < q.nv) {
                        const float y = acc[0][j] + bias;
                        // |y| bits order like |y|; NaN counts as nothing
                        const int ex = y_block_exp(__uint_as_float(
                            __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(0.f, fabsf(y))))));
                        if (ok) {
                            o[(size_t)j * a.N] = __half_as_ushort(__float2half_rn(y * exp2i(-ex)));
                            if (lane == 0) os[(size_t)j * (a.N / kYBlock)] = (int8_t)ex;
                        }
                    }
                }
            } else {
                // h = silu(gate) up: one column per thread.  Interleaved rows: lanes 2i and
                // 2i+1 hold gate and up; the even lane takes the pair of tile 0, the odd lane
                // that of tile 1.  Concatenated: tile 0 is the gates, tile 1 the ups.
                constexpr int T1 = C::kAcc - 1;
                const int hc = concat ? r : (r & 1) * 64 + (r >> 1);  // column inside the 128 of this unit
                float b0 = 0.f, b1 = 0.f;
                if (a.bias) {
                    b0 = __bfloat162float(a.bias[(size_t)q.e * a.N + wrow(q.nt, 0) + r]);
                    b1 = __bfloat162float(a.bias[(size_t)q.e * a.N + wrow(q.nt, 1) + r]);
                }
                float *mx = max_s + q4 * CN;
#pragma unroll
                for (int j = 0; j < CN; ++j) {
                    float g = acc[0][j] + b0, up = acc[T1][j] + b1;
                    if (!concat) {
                        const bool odd = r & 1;
                        const float other = __shfl_xor_sync(0xffffffffu, odd ? g : up, 1);
                        if (odd) g = other;
                        else up = other;
                    }
                    const float h = inf_to_nan(__fdividef(g, 1.0f + __expf(-g)) * up);
                    acc[0][j] = h;
                    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(amax_of(0.f, h)));
                    if (lane == 0) mx[j] = __uint_as_float(m);
                }
                q_epilogue_bar();
                if (ok) {
                    uint8_t *o = static_cast<uint8_t *>(a.out) + (size_t)q.m0 * (a.N / 2) + q.nt * 128 + hc;
                    uint8_t *os = static_cast<uint8_t *>(a.out_scale) + (size_t)q.m0 * (a.N / 256) + q.nt;
#pragma unroll
                    for (int j = 0; j < CN; ++j) {
                        if (j < q.nv) {
                            const uint32_t e = e4m3_scale_exp(
                                fmaxf(fmaxf(max_s[j], max_s[CN + j]), fmaxf(max_s[2 * CN + j], max_s[3 * CN + j])));
                            o[(size_t)j * (a.N / 2)] = (uint8_t)pack_e4m3x2(acc[0][j] * inv_scale_of_exp(e), 0.f);
                            if (tid == 0) os[(size_t)j * (a.N / 256)] = (uint8_t)e;
                        }
                    }
                }
                q_epilogue_bar();  // max_s has been read
            }
        }
    } else if (kGather) {
        // ------------------------------------------------------- row gather
        // thread g: 16-byte piece (g & 7) of rows (g >> 3) + 8 i, stored at
        // row * 128 + ((piece ^ (row & 7)) << 4) (the 128-byte swizzle)
        const int g = (int)threadIdx.x - 192;
        const int piece = g & 7, r0 = g >> 3;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (long long u = blockIdx.x; ok && u < units; u += gridDim.x) {
            const QUnit q = unit_of(u);
            const uint8_t *src[CN / 8];
#pragma unroll
            for (int i = 0; i < CN / 8; ++i) {
                const int rr = r0 + 8 * i;
                src[i] = nullptr;
                if (rr < q.nv) {
                    const int row = __ldg(a.gather + q.m0 + rr);
                    if (row >= 0 && row < a.rows) src[i] = a.a + (size_t)row * a.K + piece * 16;
                }
            }
            for (int kb = 0; kb < nk; ++kb) {
                bool w = true;
                if (lane == 0) w = mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort);
                w = __shfl_sync(0xffffffffu, w, 0);
                if (!w) {
                    ok = false;
                    break;
                }
                const uint32_t sx = base + stage * C::kStage + C::kStageW;
                const bool in = kb * kQK + piece * 16 < a.K;  // K is a multiple of 16
#pragma unroll
                for (int i = 0; i < CN / 8; ++i) {
                    const int rr = r0 + 8 * i;
                    // rows past the chunk's end feed only accumulator columns that are never
                    // stored; a row outside `a` and the K past the end are zeros
                    if (rr < q.nv)
                        cp_async_16_zfill(sx + rr * 128 + ((piece ^ (rr & 7)) << 4),
                                          src[i] && in ? src[i] + (size_t)kb * kQK : a.a, src[i] && in ? 16u : 0u);
                }
                cp_async_arrive_noinc(full_bar(stage));
                if (++stage == C::kStages) {
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
        const uint64_t t0 = globaltimer_ns();  // let copies already issued land
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::kTmem);
    }
}

template <int CN, int kMode, bool kGather>
cudaError_t launch_one(Fp8GemmArgs &a, int num_sms, cudaStream_t s) {
    using C = QCfg<CN, kMode>;
    auto *kernel = fp8_gemm_kernel<CN, kMode, kGather>;
    int unused = 0;
    cudaError_t err = launch_setup_once((const void *)kernel, &unused, [&](int, int *v) -> cudaError_t {
        *v = 1;
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    });
    if (err != cudaSuccess) return err;
    {
        const uint64_t dims[3] = {(uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.E};
        const uint64_t strides[2] = {(uint64_t)a.K, (uint64_t)a.K * a.N};
        const uint32_t box[3] = {kQK, kQM, 1};
        if (!make_map_u8(&a.tmap_w, a.w, 3, dims, strides, box))
            return cudaErrorInvalidValue;
    }
    if (!kGather) {
        const uint64_t dims[2] = {(uint64_t)a.K, (uint64_t)a.rows};
        const uint64_t strides[1] = {(uint64_t)a.K};
        const uint32_t box[2] = {kQK, CN};
        if (!make_map_u8(&a.tmap_a, a.a, 2, dims, strides, box)) return cudaErrorInvalidValue;
    }
    // no more chunks than P / CN and one begun per expert
    const int n_tiles = kMode == kFp8SwiGlu ? a.N / 256 : (a.N + kQM - 1) / kQM;
    const int64_t chunks = a.P / CN + (a.E < a.P ? a.E : a.P);
    const int64_t units = chunks * n_tiles;
    const int ctas = (int)(units < num_sms ? units : num_sms);
    return launch_maybe_pdl(kernel, dim3(ctas), dim3(kGather ? 256 : 192), C::kSmem, s, a.pdl != 0, a);
}

}  // namespace

cudaError_t launch_fp8_gemm(int mode, Fp8GemmArgs &a, int num_sms, cudaStream_t s) {
    if (a.P == 0 || a.N == 0) return cudaSuccess;
    const bool e8m0 = !a.a_f32 && !a.w_f32;
    if (a.P > 128ll * a.E)  // long segments: 256-row tiles on CTA pairs
        return e8m0 ? launch_fp8_mx_pair_gemm(mode, a, num_sms, s) : launch_fp8_pair_gemm(mode, a, num_sms, s);
    if (e8m0) return launch_fp8_few_gemm(mode, a, num_sms, s);
    // chunks of 32 rows where the segments hold no more than that on average, else large ones
    const bool few = a.P <= 32ll * a.E;
    if (mode == kFp8SwiGlu)
        return few ? launch_one<32, kFp8SwiGlu, true>(a, num_sms, s) : launch_one<64, kFp8SwiGlu, true>(a, num_sms, s);
    if (mode == kFp8Y16)
        return few ? launch_one<32, kFp8Y16, false>(a, num_sms, s) : launch_one<128, kFp8Y16, false>(a, num_sms, s);
    if (a.gather)
        return few ? launch_one<32, kFp8Bf16, true>(a, num_sms, s) : launch_one<128, kFp8Bf16, true>(a, num_sms, s);
    return few ? launch_one<32, kFp8Bf16, false>(a, num_sms, s) : launch_one<128, kFp8Bf16, false>(a, num_sms, s);
}

}  // namespace moe
