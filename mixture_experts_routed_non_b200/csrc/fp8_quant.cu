// Quantisers of the 8-bit path: rows [M,K] bf16 to e4m3 with an e8m0 scale per
// 128 values, and weights [E,K,N] bf16 (the framework's layout) to e4m3 [E,N,K]
// (K contiguous, as the tensor cores read them) with a scale per 128 x 128
// block.  Both are bound by reading bf16 and writing half as much.
#include "fp8.cuh"

namespace moe {
namespace {

// One half-warp per block of 128 values: 8 values (16 bytes) per thread.
__global__ void __launch_bounds__(256) quantize_rows_kernel(const __nv_bfloat16 *x, int64_t M, int K, int nk,
                                                            uint8_t *q, uint8_t *scale) {
    const int64_t n = M * nk;
    const int sub = threadIdx.x & 15;
    // the bound is rounded up to whole warps: every lane takes part in the shuffles
    for (int64_t b = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); b < ((n + 1) & ~1ll); b += (int64_t)gridDim.x * 16) {
        const int64_t row = b / nk;
        const int kb = (int)(b - row * nk), k = kb * kScaleBlock + sub * 8;
        const bool in = b < n && k < K;
        float f[8] = {};
        if (in) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(x + (size_t)row * K + k));
            f[0] = bf16lo(v.x), f[1] = bf16hi(v.x), f[2] = bf16lo(v.y), f[3] = bf16hi(v.y);
            f[4] = bf16lo(v.z), f[5] = bf16hi(v.z), f[6] = bf16lo(v.w), f[7] = bf16hi(v.w);
        }
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[j] = inf_to_nan(f[j]);
            m = amax_of(m, f[j]);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t e = e4m3_scale_exp(m);
        const float is = inv_scale_of_exp(e);
        if (in)
            *reinterpret_cast<uint2 *>(q + (size_t)row * K + k) =
                make_uint2(pack_e4m3x4(f[0] * is, f[1] * is, f[2] * is, f[3] * is),
                           pack_e4m3x4(f[4] * is, f[5] * is, f[6] * is, f[7] * is));
        if (b < n && sub == 0) scale[b] = (uint8_t)e;
    }
}

// One CTA per 128 x 128 block: read along N, transpose through shared memory, write along K.
__global__ void __launch_bounds__(256) quantize_weight_kernel(const __nv_bfloat16 *w, int K, int N, int nk, int nb,
                                                              uint8_t *q, uint8_t *scale) {
    __shared__ __nv_bfloat16 tile[128][130];
    __shared__ float red[8];
    const int kb = blockIdx.x, bn = blockIdx.y;
    const size_t e = blockIdx.z;
    const int k0 = kb * 128, n0 = bn * 128;
    const __nv_bfloat16 *src = w + e * (size_t)K * N;
    float m = 0.f;
    for (int i = threadIdx.x; i < 128 * 128; i += 256) {
        const int k = i >> 7, n = i & 127;
        float v = 0.f;
        if (k0 + k < K && n0 + n < N) v = inf_to_nan(__bfloat162float(src[(size_t)(k0 + k) * N + n0 + n]));
        tile[n][k] = __float2bfloat16_rn(v);  // exact: v is a bf16 or NaN
        m = amax_of(m, v);
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
    uint8_t *dst = q + e * (size_t)N * K;
    for (int i = threadIdx.x; i < 128 * 32; i += 256) {
        const int n = i >> 5, k = (i & 31) * 4;
        auto v = [&](int j) { return __bfloat162float(tile[n][k + j]) * is; };
        if (n0 + n < N && k0 + k < K)  // K is a multiple of 16: the four are all inside
            *reinterpret_cast<uint32_t *>(dst + (size_t)(n0 + n) * K + k0 + k) = pack_e4m3x4(v(0), v(1), v(2), v(3));
    }
}

}  // namespace

cudaError_t launch_quantize_rows(const __nv_bfloat16 *x, int64_t M, int32_t K, uint8_t *q, uint8_t *scale,
                                 cudaStream_t s) {
    const int nk = scale_blocks(K);
    const int64_t ctas = (M * nk + 15) / 16;
    if (ctas == 0) return cudaSuccess;
    quantize_rows_kernel<<<(unsigned)(ctas < (1 << 20) ? ctas : (1 << 20)), 256, 0, s>>>(x, M, K, nk, q, scale);
    return cudaGetLastError();
}

cudaError_t launch_quantize_weight(const __nv_bfloat16 *w, int32_t E, int32_t K, int32_t N, uint8_t *q,
                                   uint8_t *scale, cudaStream_t s) {
    const int nk = scale_blocks(K), nb = scale_blocks(N);
    quantize_weight_kernel<<<dim3(nk, nb, E), 256, 0, s>>>(w, K, N, nk, nb, q, scale);
    return cudaGetLastError();
}

}  // namespace moe
