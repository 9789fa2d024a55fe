// RMS norm with the residual's addition, in bf16 and in 8 bits, and its
// gradient.
//
//   s = bf16(x + residual)            (s = x without a residual)
//   inv = 1 / sqrt(mean_j s_j^2 + eps)
//   y_j = s_j inv w_j
//   outputs: s, y as bf16, y as e4m3 with a power-of-two scale per 128 columns, inv
//
// The norm reads the rounded sum s, which is also what it hands on as the
// residual stream, so the backward needs s and inv alone.  s_j w_j is exact in
// fp32 (two 8-bit significands); y is rounded once by the product with inv and
// once into its output type.
//
// Backward, given dy (of y) and dres (of s, from the rest of the residual
// stream, or none):
//   c = (1/H) sum_j w_j dy_j s_j
//   dx_j = dres_j + inv w_j dy_j - inv^3 c s_j       (the gradient of x and of residual alike)
//   dw_j = sum over rows of dy_j s_j inv
#include "fp8.cuh"

namespace moe {
namespace {

constexpr int kNT = 256;  // threads per row

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    f[0] = bf16lo(v.x), f[1] = bf16hi(v.x), f[2] = bf16lo(v.y), f[3] = bf16hi(v.y);
    f[4] = bf16lo(v.z), f[5] = bf16hi(v.z), f[6] = bf16lo(v.w), f[7] = bf16hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// Sum over the block, the same value in every thread.
__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();  // the previous row's sums have been read
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kNT / 32; ++i) t += red[i];
    return t;
}

// One block per row; thread t holds the 8-column chunks t, t + 256, ...
template <int V>
__global__ void __launch_bounds__(kNT) add_rmsnorm_kernel(const NormArgs a) {
    __shared__ float red[kNT / 32];
    const int chunks = a.H / 8;
    const size_t row = (size_t)blockIdx.x * a.H;
    float f[V][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * kNT;
        if (c < chunks) {
            const uint4 xv = *reinterpret_cast<const uint4 *>(a.x + row + c * 8);
            unpack8(xv, f[i]);
            if (a.residual) {
                float r[8];
                unpack8(*reinterpret_cast<const uint4 *>(a.residual + row + c * 8), r);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] += r[j];
                const uint4 sv = pack8(f[i]);
                *reinterpret_cast<uint4 *>(a.res + row + c * 8) = sv;
                unpack8(sv, f[i]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(f[i][j], f[i][j], ss);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] = 0.f;
        }
    }
    ss = block_sum(ss, red);
    const float inv = 1.0f / sqrtf(ss / (float)a.H + a.eps);
    if (a.inv_rms && threadIdx.x == 0) a.inv_rms[blockIdx.x] = inv;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * kNT;
        const bool in = c < chunks;
        float w[8] = {};
        if (in) unpack8(__ldg(reinterpret_cast<const uint4 *>(a.weight) + c), w);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = f[i][j] * w[j] * inv;
        if (a.y && in) *reinterpret_cast<uint4 *>(a.y + row + c * 8) = pack8(y);
        if (a.y8) {
            // 16 consecutive threads hold one block of 128 columns
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[j] = inf_to_nan(y[j]);
                m = amax_of(m, y[j]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const uint32_t e = e4m3_scale_exp(m);
            const float is = inv_scale_of_exp(e);
            if (in) {
                *reinterpret_cast<uint2 *>(a.y8 + row + c * 8) =
                    make_uint2(pack_e4m3x4(y[0] * is, y[1] * is, y[2] * is, y[3] * is),
                               pack_e4m3x4(y[4] * is, y[5] * is, y[6] * is, y[7] * is));
                if ((c & 15) == 0)
                    a.y8_scale[(size_t)blockIdx.x * ((a.H + kScaleBlock - 1) / kScaleBlock) + (c >> 4)] = (uint8_t)e;
            }
        }
    }
}

// Rows dealt over the blocks; each block sums its rows' dw in registers and
// leaves them in part[block].
template <int V>
__global__ void __launch_bounds__(kNT) add_rmsnorm_bwd_kernel(const NormBwdArgs a) {
    __shared__ float red[kNT / 32];
    const int chunks = a.H / 8;
    float dw[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    for (int64_t t = blockIdx.x; t < a.N; t += gridDim.x) {
        const size_t row = (size_t)t * a.H;
        const float inv = __ldg(a.inv_rms + t);
        float dy[V][8], s[V][8];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * kNT;
            if (c < chunks) {
                float w[8];
                unpack8(*reinterpret_cast<const uint4 *>(a.dy + row + c * 8), dy[i]);
                unpack8(__ldg(reinterpret_cast<const uint4 *>(a.res + row) + c), s[i]);
                unpack8(__ldg(reinterpret_cast<const uint4 *>(a.weight) + c), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dw[i][j] = fmaf(dy[i][j] * inv, s[i][j], dw[i][j]);
                    dy[i][j] *= w[j];
                    dot = fmaf(dy[i][j], s[i][j], dot);
                }
            }
        }
        dot = block_sum(dot, red);
        const float k = inv * inv * (dot / (float)a.H);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * kNT;
            if (c < chunks) {
                float d[8] = {};
                if (a.dres) unpack8(*reinterpret_cast<const uint4 *>(a.dres + row + c * 8), d);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] += inv * (dy[i][j] - s[i][j] * k);
                *reinterpret_cast<uint4 *>(a.dx + row + c * 8) = pack8(d);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * kNT;
        if (c < chunks) {
            float4 *p = reinterpret_cast<float4 *>(a.part + (size_t)blockIdx.x * a.H + c * 8);
            p[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            p[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    }
}

// dweight[c] = the sum of part[0..parts)[c], in order within each of 8 groups, then over the groups.
__global__ void __launch_bounds__(256) norm_dweight_kernel(const float *part, int parts, int H, float *dweight) {
    __shared__ float sm[8][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    float v = 0.f;
    if (c < H)
        for (int i = g; i < parts; i += 8) v += part[(size_t)i * H + c];
    sm[g][threadIdx.x & 31] = v;
    __syncthreads();
    if (g == 0 && c < H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += sm[i][threadIdx.x];
        dweight[c] = v;
    }
}

}  // namespace

int norm_bwd_parts(int64_t N) { return (int)(N < 592 ? (N > 0 ? N : 1) : 592); }

cudaError_t launch_add_rmsnorm(const NormArgs &a, int, cudaStream_t s) {
    if (a.N == 0) return cudaSuccess;
    const int v = (a.H / 8 + kNT - 1) / kNT;
    if (v <= 1) add_rmsnorm_kernel<1><<<(unsigned)a.N, kNT, 0, s>>>(a);
    else if (v <= 2) add_rmsnorm_kernel<2><<<(unsigned)a.N, kNT, 0, s>>>(a);
    else if (v <= 4) add_rmsnorm_kernel<4><<<(unsigned)a.N, kNT, 0, s>>>(a);
    else add_rmsnorm_kernel<8><<<(unsigned)a.N, kNT, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_add_rmsnorm_backward(const NormBwdArgs &a, cudaStream_t s) {
    const int parts = norm_bwd_parts(a.N);
    const int v = (a.H / 8 + kNT - 1) / kNT;
    if (v <= 1) add_rmsnorm_bwd_kernel<1><<<parts, kNT, 0, s>>>(a);
    else if (v <= 2) add_rmsnorm_bwd_kernel<2><<<parts, kNT, 0, s>>>(a);
    else if (v <= 4) add_rmsnorm_bwd_kernel<4><<<parts, kNT, 0, s>>>(a);
    else add_rmsnorm_bwd_kernel<8><<<parts, kNT, 0, s>>>(a);
    norm_dweight_kernel<<<(a.H + 31) / 32, 256, 0, s>>>(a.part, parts, a.H, a.dweight);
    return cudaGetLastError();
}

}  // namespace moe
