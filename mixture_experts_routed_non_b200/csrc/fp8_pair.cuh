// What the two CTA-pair kernels of the block-scaled products share: the tile, the
// per-expert table of row tiles, and the epilogue from a thread's 64 finished
// accumulator columns to global memory.
//
// Tile: 256 rows of one segment x 256 weight rows, on a cluster of two CTAs.  CTA
// r holds rows [128 r, 128 r + 128) of `a` and weight rows [128 r, 128 r + 128) of
// each stage of 128 K (16 KB + 16 KB); the even CTA issues the pair MMA (M = 256,
// N = 256, K = 32) for both, so each SM reads half the operand bytes per product
// that a tile of its own would need.  With SwiGLU the 256 weight rows are 128
// gates and their 128 ups.  Sixteen epilogue warps: four per TMEM lane quarter,
// 64 columns each.
#pragma once

#include "fp8.cuh"

namespace moe {

#if defined(__CUDACC__)

constexpr int kPM = 256;                    // rows per tile
constexpr int kPN = 256;                    // weight rows per tile
constexpr int kPK = 128;                    // K per stage = one scale block
constexpr uint32_t kPHalf = 128 * kPK;      // 16 KB: one CTA's share of an operand stage
constexpr uint32_t kPStage = 2 * kPHalf;
constexpr int kPGather = 128;               // gather threads of a CTA
constexpr int kPEpiWarps = 16;
constexpr uint32_t kPTmem = 512;
constexpr uint32_t kPStore = 32 * 64;       // per epilogue warp: 32 rows x 32 16-bit columns
constexpr int kPListed = 64;                // a cluster's first tiles, looked up once

template <int R>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
// The four epilogue warps that share a lane quarter's rows.
__device__ __forceinline__ void p_rows_bar(int q4) { asm volatile("bar.sync %0, 128;" ::"r"(1 + q4) : "memory"); }

// The flag (a shared address) in all CTAs of the cluster.  (Kept out of the warps' code: inlined it cost
// layers of 8 and 512 tokens 4 and 2 %.)
static __device__ __noinline__ void raise_abort(uint32_t flag, int ctas) {
    for (int c = 0; c < ctas && ctas > 1; ++c)  // (its own is up)
        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(mapa_shared(flag, (uint32_t)c)), "r"(1u) : "memory");
}
// A wait of an epilogue warp.  Where it gives up, the abort flag goes up in all CTAs of the cluster; the
// warp runs on over whatever is there and meets the barriers.  What it writes or lets others write from
// then on may be wrong, in the peers as well.  So every CTA looks at its flag once the whole cluster is
// through, and writes NaN over its output where it is up.  (Nothing is added where a wait succeeds: a note
// of each wait's result, or a vote on it, cost 3-6 % of the products with fp32 scales, a third of 1001 x
// 2000 x 1496.)
__device__ __forceinline__ void epi_wait(uint32_t bar, uint32_t parity, volatile uint32_t *abort, int ctas,
                                         unsigned long long timeout_ns = kWaitTimeoutNs) {
    if (!mbar_wait_bounded(bar, parity, abort, timeout_ns)) raise_abort(smem_u32(const_cast<const uint32_t *>(abort)), ctas);
}

// Four floats of another CTA's shared memory.
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t cluster_addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}

struct PTile {
    int e, nt, m0, m_end;
};

// The tile list: row tiles expert by expert, each row tile's weight tiles together
// (neighbouring clusters share its rows in L2).  off_s and pre_s are shared-memory
// tables of E + 1 entries, first a table of the cluster's first kPListed tiles: a look-up
// takes some 900 clocks beside the other warps, and every role needs every tile (with 2
// blocks of K a tile takes 3500).  kOne: one segment of all P rows, no tables.
template <bool kOne>
struct PTiles {
    const int *off_s, *pre_s;
    int4 *first;
    int listed;  // its size: 0 where tiles are few
    int E, N, n_tiles, P;
    bool concat;
    __device__ __forceinline__ int count() const {  // below 2^31 (fp8_sizes_ok)
        return (kOne ? (P + kPM - 1) / kPM : pre_s[E]) * n_tiles;
    }
    // by all threads of the block; t0, dt: the cluster's tiles
    __device__ __forceinline__ void fill(int t0, int dt) {
        if (kOne) return;
        const int n = count(), i = (int)threadIdx.x;
        listed = n > 2 * dt ? kPListed : 0;
        if (listed == 0) return;
        if (i < kPListed && t0 + i * dt < n) {
            const PTile t = find(t0 + i * dt);
            first[i] = make_int4(t.e, t.nt, t.m0, t.m_end);
        }
        __syncthreads();
    }
    // tile u, the cluster's i-th
    __device__ __forceinline__ PTile at(int u, int i) const {
        if (kOne || i >= listed) return find(u);
        const int4 v = first[i];
        PTile t;
        t.e = v.x, t.nt = v.y, t.m0 = v.z, t.m_end = v.w;
        return t;
    }
    __device__ __forceinline__ PTile find(int u) const {
        PTile t;
        const int mt = u / n_tiles;
        t.nt = u - mt * n_tiles;
        if (kOne) {
            t.e = 0, t.m0 = mt * kPM, t.m_end = P;
            return t;
        }
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
    }
    // first weight row of half h (accumulator columns 128 h ..) of a tile
    __device__ __forceinline__ int wrow(int nt, int h) const {
        return concat ? h * (N / 2) + nt * 128 : nt * kPN + h * 128;
    }
};

// Segment offsets into off_s, held inside [0, P] whatever the caller's table says.
__device__ __forceinline__ void load_offsets(const Fp8GemmArgs &a, int *off_s, int threads) {
    for (int i = threadIdx.x; i <= a.E; i += threads)
        off_s[i] = (int)min(max((long long)load_now(a.expert_off + i), 0ll), (long long)a.P);
}
// pre_s[e] = pieces of `rows` rows in the experts below e (one converged warp).  Held at
// the most that ascending offsets can give: a table that goes up and down would count
// rows again and again, past what fp8_sizes_ok has bounded.  (No overflow before the
// minimum: of 32 differences inside [0, P] no more than 16 can be P.)
__device__ __forceinline__ void prefix_pieces(const int *off_s, int *pre_s, int E, int64_t P, int rows, int lane) {
    const int most = (int)(P / rows + (E < P ? E : P));
    int sum = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        const int n = e < E ? (max(off_s[e + 1] - off_s[e], 0) + rows - 1) / rows : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (e < E) pre_s[e] = min(sum + incl - n, most);
        sum = min(sum + __shfl_sync(0xffffffffu, incl, 31), most);
    }
    if (lane == 0) pre_s[E] = sum;
}

// 32 16-bit columns (16 packed pairs) of one row per lane: a warp whose 32 rows
// are all stored goes through shared memory (64-byte swizzle) and one TMA store
// (columns past N are clipped); otherwise each valid lane stores its row.
__device__ __forceinline__ void store32(const CUtensorMap *map, uint32_t buf, int lane, bool warp_full, bool valid,
                                        int row0, uint16_t *row, int col0, int N, const uint32_t (&v)[16]) {
    if (warp_full) {
        if (lane == 0) bulk_wait_read0();  // the buffer's previous store has been read
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c)
            st_shared_v4(buf + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4), v[4 * c], v[4 * c + 1], v[4 * c + 2],
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
        for (int c = 0; c < 4; ++c)
            if (col0 + 8 * c < N) dst[c] = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    }
}

// The row gather of one CTA's stages, by 128 threads: thread g copies the 16-byte
// piece (g & 7) of rows (g >> 3) + 16 i to row * 128 + ((piece ^ (row & 7)) << 4)
// (the 128-byte swizzle).  Rows past the segment's end feed only accumulator rows
// that are never stored and are not copied.  Every copy reads a valid address
// unconditionally -- a row outside `a` some other row (pair_output drops what it
// gave), a piece past the end of K the row's last one (the weights are zeros
// there) -- because a choice between two sources, or the copy's own zero fill,
// cost a quarter to a half of the whole product (131072 x 2048 x 1536 over 128
// experts, when it was tried: 358 us like this, 465 with a zero row, 547 with zero fill).
template <int kStages, typename Empty, typename Gfull>
__device__ __forceinline__ void gather_rows(const Fp8GemmArgs &a, const PTiles<false> &list, int rank, int g, uint32_t base,
                                            Empty empty_bar, Gfull gfull_bar, volatile uint32_t *abort, int t0,
                                            int dt) {
    const int piece = g & 7, r0 = g >> 3;
    const int tiles = list.count();
    int stage = 0;
    uint32_t phase = 0;
    for (int u = t0, i = 0; u < tiles; u += dt, ++i) {
        const PTile t = list.at(u, i);
        int row[8];  // -1: not copied
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int p = t.m0 + rank * 128 + r0 + 16 * i;
            row[i] = p < t.m_end ? (int)min((long long)max(load_now(a.gather + p), 0), (long long)a.rows - 1) : -1;
        }
        for (int kb = 0; kb < a.nk; ++kb) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort))) {
                cp_async_wait_all();
                return;
            }
            const uint32_t dst = base + stage * kPStage + r0 * 128 + ((piece ^ (r0 & 7)) << 4);
            const uint8_t *src = a.a + min(kb * kPK + piece * 16, a.K - 16);  // K is a multiple of 16
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (row[i] >= 0) cp_async_16(dst + i * 2048, src + (size_t)row[i] * a.K);
            cp_async_arrive_noinc(gfull_bar(stage));
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
    cp_async_wait_all();
}

// A tile whose K is shared by kSplit pairs, a cluster: each pair has the sums of its part of K.
// The pairs share out the columns; each adds the others' sums of its columns, left in shared
// memory in the place of the ring (whose last MMA has read it), in pair order.  False: this
// warp's columns are another pair's.  All threads of the cluster meet in it once, those of
// other warps in a cluster_sync_all() of their own.
template <int kSplit>
__device__ __forceinline__ bool pair_share(float (&acc)[64], uint32_t ring, int rank, int pi, int cq, int q4, int lane) {
    const bool mine = cq * kSplit / 4 == pi;
    // [cq][16 groups of four columns][128 rows][4]
    const uint32_t part = ring + (uint32_t)cq * 32768u + (uint32_t)(32 * q4 + lane) * 16u;
    if (!mine) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            st_shared_v4(part + j * 2048u, __float_as_uint(acc[4 * j]), __float_as_uint(acc[4 * j + 1]),
                         __float_as_uint(acc[4 * j + 2]), __float_as_uint(acc[4 * j + 3]));
    }
    __syncwarp();
    cluster_sync_all();
    if (!mine) return false;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int p = 0; p < kSplit; ++p) {
            float4 v = make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
            if (p != pi) v = ld_cluster_f4(mapa_shared(part + j * 2048u, (uint32_t)(2 * p + rank)));
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        acc[4 * j] = s.x, acc[4 * j + 1] = s.y, acc[4 * j + 2] = s.z, acc[4 * j + 3] = s.w;
    }
    return true;
}

// v[0, 8) += the eight biases from `b` on: one load where they are aligned (aligned is
// uniform).
__device__ __forceinline__ void add_bias8(const __nv_bfloat16 *b, bool aligned, float *v) {
    if (aligned) {
        const uint4 w = *reinterpret_cast<const uint4 *>(b);
        v[0] += bf16lo(w.x), v[1] += bf16hi(w.x), v[2] += bf16lo(w.y), v[3] += bf16hi(w.y);
        v[4] += bf16lo(w.z), v[5] += bf16hi(w.z), v[6] += bf16lo(w.w), v[7] += bf16hi(w.w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += __bfloat162float(b[i]);
    }
}
// (every row and every eighth column of [E, N] keeps the base's alignment: N is a multiple of 8)
__device__ __forceinline__ bool bias_aligned(const Fp8GemmArgs &a) {
    return (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0;
}

// One epilogue thread's part of a finished tile: row r of this CTA's 128 and 64
// accumulator columns acc -- the tile's columns [64 cq, 64 cq + 64), or, with
// concatenated SwiGLU, gates [32 cq, 32 cq + 32) and their ups.  buf: the warp's
// store buffer; max_s: [4][128] row maxima (SwiGLU), the other of two at the next tile, by whose
// barrier these have been read.  All 16 warps call it.
template <int kMode, bool kGather>
__device__ __forceinline__ void pair_output(const Fp8GemmArgs &a, const PTile &t, float (&acc)[64], int rank, int cq,
                                            int q4, int lane, bool concat, uint32_t buf, float *max_s) {
    const int r = 32 * q4 + lane;
    const int row0 = t.m0 + rank * 128 + q4 * 32;
    const int p = row0 + lane;
    const bool store = p < t.m_end;
    if (kGather && p < t.m_end) {  // a gathered row outside `a` counts as zeros
        const int src = load_now(a.gather + p);
        if (src < 0 || src >= a.rows) {
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = 0.f;
        }
    }
    if (kMode != kFp8SwiGlu) {
        const int col = t.nt * kPN + cq * 64;
        if (col < a.N) {
            if (a.bias) {
                const __nv_bfloat16 *br = a.bias + (size_t)t.e * a.N + col;
                const bool al = bias_aligned(a);
#pragma unroll
                for (int j = 0; j < 64; j += 8)
                    if (col + j < a.N) add_bias8(br + j, al, acc + j);
            }
            if (kMode == kFp8Y16) {  // fp16 scaled by a power of two per 32 columns
                uint32_t exps = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float m = 0.f;
#pragma unroll
                    for (int j = 0; j < 32; ++j) m = amax_of(m, acc[32 * i + j]);
                    const int ex = y_block_exp(m);
                    const float sc = exp2i(-ex);
                    exps |= (uint32_t)(uint8_t)(int8_t)ex << (8 * i);
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[32 * i + j] *= sc;
                }
                if (store)  // N is a multiple of 128: the two exponents are one aligned half-word
                    *reinterpret_cast<uint16_t *>(static_cast<int8_t *>(a.out_scale) +
                                                  (size_t)p * (a.N / kYBlock) + col / kYBlock) = (uint16_t)exps;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v[j] = kMode == kFp8Y16 ? pack_f16x2(acc[32 * i + 2 * j], acc[32 * i + 2 * j + 1])
                                            : pack_bf16x2(acc[32 * i + 2 * j], acc[32 * i + 2 * j + 1]);
                if (col + 32 * i < a.N)
                    store32(&a.tmap_out, buf, lane, row0 + 31 < t.m_end, store, row0,
                            static_cast<uint16_t *>(a.out) + (size_t)(store ? p : 0) * a.N, col + 32 * i, a.N, v);
            }
        }
    } else {
        // h = silu(gate) up: 32 columns per thread, with the other three quarters' one scale block
        const int hc = t.nt * 128 + cq * 32;  // first h column of this thread
        if (a.bias) {
            const __nv_bfloat16 *br = a.bias + (size_t)t.e * a.N;
            const bool al = bias_aligned(a);
#pragma unroll
            for (int j = 0; j < 64; j += 8)
                add_bias8(br + (concat ? (j < 32 ? hc + j : a.N / 2 + hc + j - 32) : 2 * hc + j), al, acc + j);
        }
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            // interleaved: columns 2j, 2j+1; the value goes to acc[j], whose own column
            // has been used by then (j <= 2j)
            const float g = concat ? acc[j] : acc[2 * j], up = concat ? acc[32 + j] : acc[2 * j + 1];
            const float h = inf_to_nan(__fdividef(g, 1.0f + __expf(-g)) * up);
            acc[j] = h;
            m = amax_of(m, h);
        }
        max_s[cq * 128 + r] = m;
        p_rows_bar(q4);
        m = fmaxf(fmaxf(max_s[r], max_s[128 + r]), fmaxf(max_s[256 + r], max_s[384 + r]));
        const uint32_t e = e4m3_scale_exp(m);
        const float is = inv_scale_of_exp(e);
        if (store) {
            uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.out) + (size_t)p * (a.N / 2) + hc);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = 16 * i + 4 * k;
                    v[k] = pack_e4m3x4(acc[j] * is, acc[j + 1] * is, acc[j + 2] * is, acc[j + 3] * is);
                }
                o[i] = make_uint4(v[0], v[1], v[2], v[3]);
            }
            if (cq == 0) static_cast<uint8_t *>(a.out_scale)[(size_t)p * (a.N / 256) + t.nt] = (uint8_t)e;
        }
    }
}

// NaN into `bytes` bytes of output (a multiple of 8, aligned to it): all ones but the signs, in each of the types.
template <int kMode>
__device__ __forceinline__ void store_nan(uint8_t *out, int bytes) {
    const uint32_t v = kMode == kFp8SwiGlu ? 0x7F7F7F7Fu : 0x7FFF7FFFu;
    for (int i = 0; i < bytes; i += 8) *reinterpret_cast<uint2 *>(out + i) = make_uint2(v, v);
}
// NaN over an epilogue warp's part of all of the cluster's tiles (epi_wait).
template <int kMode, bool kOne>
__device__ __forceinline__ void nan_tiles(const Fp8GemmArgs &a, const PTiles<kOne> &list, int tiles, int t0, int dt, int rank,
                                          int cq, int q4, int lane) {
    for (int u = t0, i = 0; u < tiles; u += dt, ++i) {
        const PTile t = list.at(u, i);
        const int p = t.m0 + rank * 128 + q4 * 32 + lane;
        const int col = kMode == kFp8SwiGlu ? t.nt * 128 + cq * 32 : t.nt * kPN + cq * 64;
        const int row_bytes = kMode == kFp8SwiGlu ? a.N / 2 : 2 * a.N, size = kMode == kFp8SwiGlu ? 1 : 2;
        if (p < t.m_end)
            store_nan<kMode>(static_cast<uint8_t *>(a.out) + (size_t)p * row_bytes + (size_t)col * size,
                             min(kMode == kFp8SwiGlu ? 32 : 128, row_bytes - col * size));
    }
}

#endif  // __CUDACC__

}  // namespace moe
