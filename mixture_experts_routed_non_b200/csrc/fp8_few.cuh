// What the two kernels for segments of a few rows share: the unit list, the K split
// over a cluster, and the epilogue from partial sums in shared memory to global
// memory.
//
// Operands swapped: 128 weight rows on the MMA's M side, a chunk of up to CN rows of
// `a` on its N side, so that a tile's arithmetic follows the few rows there are (N is
// always CN: what lies behind the chunk's rows is never read back).  With SwiGLU a
// unit has two weight tiles (256 rows: 128 columns of h).
//
// Few units: a cluster of S CTAs shares a unit, each taking 1/S of K, so that all
// SMs pull on memory even when one token meets one matrix.  Each CTA leaves its
// partial sums in its shared memory; the CTAs then share out the tokens, and each
// adds the S partial sums of its tokens in rank order (no atomics: the result does
// not depend on timing) and writes them.
#pragma once

#include "fp8_pair.cuh"

namespace moe {

constexpr int kFM = 128;                  // weight rows per MMA
constexpr int kFMaxSplit = 8;

#if defined(__CUDACC__)

constexpr uint32_t kFTileW = kFM * kPK;   // 16 KB
constexpr int kFGather = 64;              // gather threads
constexpr int kFListed = 64;              // a CTA's first units, looked up once

// Cluster-scope release and acquire: shared-memory data handed to another CTA.
__device__ __forceinline__ void mbar_arrive_cluster_release(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void fence_acquire_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

struct FUnit {
    int e, nt, m0, nv;  // expert, weight tile, first sorted position, rows
};

// Units: experts in order, inside one its weight tiles, inside a tile its chunks.
// off_s and pre_s (chunks below each expert) are shared-memory tables of E + 1, first one
// of the CTA's first kFListed units (as in PTiles).  kOne: one segment, no tables.
template <int CN, int kMode, bool kOne>
struct FUnits {
    const int *off_s, *pre_s;
    int4 *first;
    int listed;
    int E, N, n_tiles, P;
    bool concat;
    __device__ __forceinline__ void fill(int units, int u0, int du) {
        if (kOne) return;
        const int i = (int)threadIdx.x;
        listed = units > 2 * du ? kFListed : 0;
        if (listed == 0) return;
        if (i < kFListed && u0 + i * du < units) {
            const FUnit q = find(u0 + i * du);
            first[i] = make_int4(q.e, q.nt, q.m0, q.nv);
        }
        __syncthreads();
    }
    // unit u, the CTA's i-th
    __device__ __forceinline__ FUnit at(int u, int i) const {
        if (kOne || i >= listed) return find(u);
        const int4 v = first[i];
        FUnit q;
        q.e = v.x, q.nt = v.y, q.m0 = v.z, q.nv = v.w;
        return q;
    }
    __device__ __forceinline__ FUnit find(int u) const {
        if (kOne) {
            const int ch = (P + CN - 1) / CN;
            FUnit q;
            q.e = 0;
            q.nt = ch == 1 ? u : u / ch;
            q.m0 = (u - q.nt * ch) * CN;
            q.nv = min(CN, P - q.m0);
            return q;
        }
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
    }
    // first weight row of tile t (0 or 1) of a unit
    __device__ __forceinline__ int wrow(int nt, int t) const {
        if (kMode != kFp8SwiGlu) return nt * kFM;
        return concat ? t * (N / 2) + nt * kFM : nt * 2 * kFM + t * kFM;
    }
};

// The row gather of one CTA's stages, by 64 threads: thread g copies the 16-byte
// piece (g & 7) of rows (g >> 3) + 8 i to row * 128 + ((piece ^ (row & 7)) << 4) (the
// 128-byte swizzle) of each stage's rows; sources as in fp8_pair.cuh.
template <int CN, int kMode, int kStages, uint32_t kStage, uint32_t kStageW, typename Empty, typename Gfull>
__device__ __forceinline__ void gather_chunk_rows(const Fp8GemmArgs &a, const FUnits<CN, kMode, false> &list, int units, int u0,
                                                  int du, int kb0, int kb1, int g, uint32_t base, Empty empty_bar,
                                                  Gfull gfull_bar, volatile uint32_t *abort) {
    const int piece = g & 7, r0 = g >> 3;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = u0, n = 0; ok && u < units; u += du, ++n) {
        const FUnit q = list.at(u, n);
        int row[CN / 8];  // -1: not copied
#pragma unroll
        for (int i = 0; i < CN / 8; ++i)
            row[i] = r0 + 8 * i < q.nv ? (int)min((long long)max(load_now(a.gather + q.m0 + r0 + 8 * i), 0),
                                                  (long long)a.rows - 1)
                                       : -1;
        for (int kb = kb0; kb < kb1; ++kb) {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort));
            if (!ok) break;
            const uint32_t dst = base + stage * kStage + kStageW + r0 * 128 + ((piece ^ (r0 & 7)) << 4);
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

// Hands this warp's partial sums over and waits for everybody's.
__device__ __forceinline__ void partials_ready(uint32_t rfull_bar, uint32_t parity, int S, int lane,
                                               volatile uint32_t *abort,
                                               unsigned long long timeout_ns = kWaitTimeoutNs) {
    __syncwarp();
    if (S == 1) {
        if (lane == 0) mbar_arrive(rfull_bar);
    } else if (lane < S) {
        mbar_arrive_cluster_release(mapa_shared(rfull_bar, lane));
    }
    epi_wait(rfull_bar, parity, abort, S, timeout_ns);
    if (S > 1) fence_acquire_cluster();
    __syncwarp();
}
// This warp has read what it needed of everybody's.
__device__ __forceinline__ void partials_read(uint32_t rempty_bar, int S, int lane) {
    __syncwarp();
    if (S == 1) {
        if (lane == 0) mbar_arrive(rempty_bar);
    } else if (lane < S) {
        mbar_arrive_cluster_release(mapa_shared(rempty_bar, lane));
    }
}

// Which of a unit's rows are gathered from outside `a`.  The sources are loaded before the
// wait for the accumulator, which hides it, and looked at behind it.
template <int CN>
struct FGone {
    int src[CN / 32];
    uint32_t bits[CN / 32];
    __device__ __forceinline__ void load(const Fp8GemmArgs &a, const FUnit &q, int lane) {
#pragma unroll
        for (int i = 0; i < CN / 32; ++i) src[i] = 32 * i + lane < q.nv ? load_now(a.gather + q.m0 + 32 * i + lane) : 0;
    }
    __device__ __forceinline__ void look(const Fp8GemmArgs &a) {
#pragma unroll
        for (int i = 0; i < CN / 32; ++i) bits[i] = __ballot_sync(0xffffffffu, src[i] < 0 || src[i] >= a.rows);
    }
};

// The unit's output for the tokens of this CTA, by 128 threads (tid).  red (its
// shared-memory address; red_ptr the same): [tile][token][weight row] fp32 in each of
// the S CTAs.
template <int CN, int kMode, bool kGather>
__device__ __forceinline__ void few_output(const Fp8GemmArgs &a, const FUnit &q, int rank, int S, int tid, bool concat,
                                           uint32_t red, const uint8_t *red_ptr, const FGone<CN> &gone) {
    constexpr int kAcc = kMode == kFp8SwiGlu ? 2 : 1;
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
                    x = *reinterpret_cast<const float4 *>(red_ptr + at);
                    y = *reinterpret_cast<const float4 *>(red_ptr + at + 16);
                }
                v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
                v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
            }
        };
        auto bias8 = [&](int col, float (&v)[8]) {
            if (a.bias) add_bias8(a.bias + (size_t)q.e * a.N + col, bias_aligned(a), v);
        };
        const size_t p = (size_t)q.m0 + jj;
        const bool outside = kGather && (gone.bits[jj >> 5] >> (jj & 31) & 1);  // counts as zeros
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
            if (n < a.N) bias8(n, v);
            if (kMode == kFp8Bf16) {
                if (has && n < a.N)
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
                if (has) {
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
                sum8(kAcc - 1, c8, up);
                keep(g);
                keep(up);
                bias8(q.nt * 128 + c8, g);
                bias8(a.N / 2 + q.nt * 128 + c8, up);
            } else {
                float x[8], y[8];
                const int t = c8 >> 6, row = 2 * (c8 & 63);
                sum8(t, row, x);
                sum8(t, row + 8, y);
                keep(x);
                keep(y);
                bias8(q.nt * 256 + 2 * c8, x);
                bias8(q.nt * 256 + 2 * c8 + 8, y);
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
            if (has) {
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + p * (a.N / 2) + q.nt * 128 + c8) =
                    make_uint2(pack_e4m3x4(g[0] * is, g[1] * is, g[2] * is, g[3] * is),
                               pack_e4m3x4(g[4] * is, g[5] * is, g[6] * is, g[7] * is));
                if ((tid & 15) == 0)
                    static_cast<uint8_t *>(a.out_scale)[p * (a.N / 256) + q.nt] = (uint8_t)e;
            }
        }
    }
}

// nan_tiles for the few-row kernels: the tokens of this CTA in all of its units.
template <int CN, int kMode, bool kOne>
__device__ __forceinline__ void nan_units(const Fp8GemmArgs &a, const FUnits<CN, kMode, kOne> &list, int units, int u0, int du,
                                          int rank, int S, int tid) {
    for (int u = u0, n = 0; u < units; u += du, ++n) {
        const FUnit q = list.at(u, n);
        const int col = q.nt * kFM + (tid & 15) * 8;  // (of h, with SwiGLU)
        if (col >= (kMode == kFp8SwiGlu ? a.N / 2 : a.N)) continue;
        for (int j = rank + (tid >> 4) * S; j < q.nv; j += 8 * S) {
            const size_t p = (size_t)q.m0 + j;
            store_nan<kMode>(static_cast<uint8_t *>(a.out) + (kMode == kFp8SwiGlu ? p * (a.N / 2) + col : 2 * (p * a.N + col)),
                             kMode == kFp8SwiGlu ? 8 : 16);
        }
    }
}

// Tensor maps of the weights and, unless they are gathered, the rows in chunks of cn.
inline bool make_few_maps(Fp8GemmArgs &a, int cn, bool rows) {
    const uint64_t wd[3] = {(uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.E};
    const uint64_t ws[2] = {(uint64_t)a.K, (uint64_t)a.K * a.N};
    const uint32_t wb[3] = {kPK, kFM, 1};
    if (!make_map_u8(&a.tmap_w, a.w, 3, wd, ws, wb)) return false;
    const uint64_t ad[2] = {(uint64_t)a.K, (uint64_t)a.rows}, as[1] = {(uint64_t)a.K};
    const uint32_t ab[2] = {kPK, (uint32_t)cn};
    return !rows || make_map_u8(&a.tmap_a, a.a, 2, ad, as, ab);
}

inline cudaLaunchAttribute few_cluster(int S) {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)S;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    return at;
}
// A few-row kernel's shared memory, and how many clusters of 2, 4 and 8 CTAs run at
// once (a byte each): one to an SM, but a cluster's SMs have to be neighbours.
inline cudaError_t few_setup(void (*kernel)(Fp8GemmArgs), int threads, size_t smem, int *clusters) {
    return launch_setup_once((const void *)kernel, clusters, [&](int, int *v) -> cudaError_t {
        cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        *v = 0;
        for (int i = 0, S = 2; err == cudaSuccess && S <= kFMaxSplit; ++i, S *= 2) {
            cudaLaunchAttribute at = few_cluster(S);
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(S);
            cfg.blockDim = dim3(threads);
            cfg.dynamicSmemBytes = smem;
            cfg.attrs = &at;
            cfg.numAttrs = 1;
            int n = 0;
            err = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
            *v |= (n < 255 ? n : 255) << (8 * i);
        }
        return err;
    });
}

// CTAs to a unit: K is split while all clusters still run at once and each CTA keeps a
// group of four blocks.  A cluster too many waits for a whole unit: 128 x 7168 x 512 in 16
// clusters of eight, of which 15 run at once, 19.0 us, in clusters of four 10.3; 96 x
// 2048 x 1536 in 36 clusters of four, of which 33, 14.1 us, of two 8.6.
inline int few_split(int64_t units, int nk, int fit) {
    int S = 1;
    for (int i = 0; S < kFMaxSplit && units <= ((fit >> (8 * i)) & 255) && nk >= 8 * S; ++i) S *= 2;
    return S;
}

// Units of chunks of cn rows: of one segment; else the most there can be (no more than P / cn chunks and one
// begun per expert).
inline int64_t few_units(int mode, const Fp8GemmArgs &a, int cn) {
    const int64_t chunks = a.expert_off ? a.P / cn + (a.E < a.P ? a.E : a.P) : (a.P + cn - 1) / cn;
    return chunks * (mode == kFp8SwiGlu ? a.N / (2 * kFM) : (a.N + kFM - 1) / kFM);
}

// Launches a few-row kernel with chunks of cn rows on as many CTAs as there can be
// units, split over K where there are few.
inline cudaError_t launch_few(void (*kernel)(Fp8GemmArgs), int mode, Fp8GemmArgs &a, int cn, int threads, size_t smem,
                              int num_sms, cudaStream_t s) {
    int fit = 0;
    const cudaError_t err = few_setup(kernel, threads, smem, &fit);
    if (err != cudaSuccess) return err;
    const int64_t units = few_units(mode, a, cn);
    const int S = few_split(units, a.nk, fit);
    a.split = S;
    int64_t clusters = num_sms / S;
    if (clusters > units) clusters = units;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * S));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (a.pdl) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (S > 1) {
        attr[cfg.numAttrs++] = few_cluster(S);
    }
    return cudaLaunchKernelEx(&cfg, kernel, (Fp8GemmArgs)a);
}

#endif  // __CUDACC__

}  // namespace moe
