// Quantisers of the 8-bit path: rows [M,K] bf16 to e4m3 with an e8m0 scale per
// 128 values, and weights [E,K,N] bf16 (the framework's layout) to e4m3 [E,N,K]
// (K contiguous, as the tensor cores read them) with a scale per 128 x 128
// block.  Both are bound by HBM, reading bf16 and writing half as much: every
// thread has 64 (rows) or 128 bytes (weights) of loads in flight before it needs one.
// Measured, launch included: rows 16384 x 7168 61 us (5.8 TB/s; with one load per thread
// 85), 16384 x 2048 22; weights 128 x 2048 x 1536 195 us (6.2 TB/s; with two-byte
// loads and a transpose in bf16 428).
#include "fp8.cuh"

namespace moe {
namespace {

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    f[0] = inf_to_nan(bf16lo(v.x)), f[1] = inf_to_nan(bf16hi(v.x)), f[2] = inf_to_nan(bf16lo(v.y));
    f[3] = inf_to_nan(bf16hi(v.y)), f[4] = inf_to_nan(bf16lo(v.z)), f[5] = inf_to_nan(bf16hi(v.z));
    f[6] = inf_to_nan(bf16lo(v.w)), f[7] = inf_to_nan(bf16hi(v.w));
}

// One half-warp per block of 128 values, 8 values (16 bytes) per thread; kRowsU blocks per
// half-warp, 16 apart.
constexpr int kRowsU = 4;
__global__ void __launch_bounds__(256) quantize_rows_kernel(const __nv_bfloat16 *x, int64_t n, int K, int nk, uint8_t *q,
                                                            uint8_t *scale) {
    const int sub = threadIdx.x & 15;
    const int64_t b0 = (int64_t)blockIdx.x * (16 * kRowsU) + (threadIdx.x >> 4);
    pdl_wait();
    pdl_launch_dependents();
    const bool whole = nk * kScaleBlock == K;  // then block b starts at value 128 b
    size_t at[kRowsU];
    uint4 v[kRowsU];
    bool in[kRowsU];
#pragma unroll
    for (int i = 0; i < kRowsU; ++i) {
        const int64_t b = b0 + 16 * i;
        in[i] = b < n;
        if (whole) {
            at[i] = (size_t)b * kScaleBlock + sub * 8;
        } else {
            const int64_t row = b / nk;
            const int k = (int)(b - row * nk) * kScaleBlock + sub * 8;
            in[i] = in[i] && k < K;
            at[i] = (size_t)row * K + k;
        }
        v[i] = in[i] ? *reinterpret_cast<const uint4 *>(x + at[i]) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kRowsU; ++i) {
        float f[8], m = 0.f;
        unpack8(v[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = amax_of(m, f[j]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t e = e4m3_scale_exp(m);
        const float is = inv_scale_of_exp(e);
        if (in[i])
            *reinterpret_cast<uint2 *>(q + at[i]) =
                make_uint2(pack_e4m3x4(f[0] * is, f[1] * is, f[2] * is, f[3] * is),
                           pack_e4m3x4(f[4] * is, f[5] * is, f[6] * is, f[7] * is));
        if (in[i] && sub == 0) scale[b0 + 16 * i] = (uint8_t)e;
    }
}

// One CTA per 128 x 128 block.  Thread (g, l) = (tid / 16, tid % 16) reads columns 8 l .. 8 l + 7
// of rows 4 g .. 4 g + 3 and 64 more, so that it holds four neighbouring k of a column: one
// word of the transposed block, which passes through shared memory.  Word (n, k / 4) sits at
// [n][(k / 4) ^ 2 (n / 8)]: a warp's 32 words of a store are in 32 banks, and pairs of
// words stay pairs for the reads along K.
__global__ void __launch_bounds__(256) quantize_weight_kernel(const __nv_bfloat16 *w, int K, int N, int nk, int nb,
                                                              uint8_t *q, uint8_t *scale) {
    __shared__ __align__(16) uint32_t tile[128][32];
    __shared__ float red[8];
    const int kb = blockIdx.x, bn = blockIdx.y;
    const size_t e = blockIdx.z;
    const int k0 = kb * 128, n0 = bn * 128;
    const int l = threadIdx.x & 15, g = threadIdx.x >> 4;
    const __nv_bfloat16 *src = w + e * (size_t)K * N + n0 + 8 * l;
    const bool in_n = n0 + 8 * l < N;  // N is a multiple of 8, K of 16
    uint4 v[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + 64 * i + 4 * g + j;
            v[i][j] = in_n && k < K ? __ldg(reinterpret_cast<const uint4 *>(src + (size_t)k * N)) : make_uint4(0, 0, 0, 0);
        }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float f[8];
            unpack8(v[i][j], f);
#pragma unroll
            for (int c = 0; c < 8; ++c) m = amax_of(m, f[c]);
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
    const uint32_t ex = e4m3_scale_exp(m);
    const float is = inv_scale_of_exp(ex);
    if (threadIdx.x == 0) scale[(e * nb + bn) * nk + kb] = (uint8_t)ex;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float f[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) unpack8(v[i][j], f[j]);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            tile[8 * l + c][(g + 16 * i) ^ (2 * l)] = pack_e4m3x4(f[0][c] * is, f[1][c] * is, f[2][c] * is, f[3][c] * is);
    }
    __syncthreads();
    uint8_t *dst = q + (e * N + n0) * (size_t)K + k0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = 16 * i + g;
        if (n0 + n < N && k0 + 8 * l < K)
            *reinterpret_cast<uint2 *>(dst + (size_t)n * K + 8 * l) =
                *reinterpret_cast<const uint2 *>(&tile[n][(2 * l) ^ (2 * (n >> 3))]);
    }
}

}  // namespace

cudaError_t launch_quantize_rows(const __nv_bfloat16 *x, int64_t M, int32_t K, uint8_t *q, uint8_t *scale,
                                 cudaStream_t s) {
    const int nk = scale_blocks(K);
    const int64_t n = M * nk, ctas = (n + 16 * kRowsU - 1) / (16 * kRowsU);
    if (ctas == 0) return cudaSuccess;
    return launch_maybe_pdl(quantize_rows_kernel, dim3((unsigned)ctas), dim3(256), 0, s, true, x, n, K, nk, q, scale);
}

cudaError_t launch_quantize_weight(const __nv_bfloat16 *w, int32_t E, int32_t K, int32_t N, uint8_t *q,
                                   uint8_t *scale, cudaStream_t s) {
    const int nk = scale_blocks(K), nb = scale_blocks(N);
    quantize_weight_kernel<<<dim3(nk, nb, E), 256, 0, s>>>(w, K, N, nk, nb, q, scale);
    return cudaGetLastError();
}

}  // namespace moe
