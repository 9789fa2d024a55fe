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

constexpr int kNMaxT = 512;  // threads per row at most

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    f[0] = bf16lo(v.x), f[1] = bf16hi(v.x), f[2] = bf16lo(v.y), f[3] = bf16hi(v.y);
    f[4] = bf16lo(v.z), f[5] = bf16hi(v.z), f[6] = bf16lo(v.w), f[7] = bf16hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// Sum over the T threads of one row (T = blockDim.x: 16, or a multiple of 32),
// the same value in each.  red: this row's kNMaxT / 32 floats; a caller that
// comes again passes another buffer in between, so that one barrier is enough.
__device__ __forceinline__ float row_sum(float v, float *red) {
    const int T = blockDim.x;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (T == 16) return v;
    v += __shfl_xor_sync(0xffffffffu, v, 16);
    if (T == 32) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < T / 32; ++i) t += red[i];
    return t;
}

// Thread (x, y) of a block works on row y of the block's rows, on the 8-column
// chunks x, x + T, ... (V of them).  A block takes rows until there are none; the
// next rows' loads are in flight while the current ones are reduced and written.
template <int V>
__global__ void __launch_bounds__(kNMaxT) add_rmsnorm_kernel(const NormArgs a) {
    __shared__ float red[2][kNMaxT / 32];
    const int T = blockDim.x, chunks = a.H / 8;
    const int blocks = (a.H + kScaleBlock - 1) / kScaleBlock;
    float *my_red[2] = {red[0] + threadIdx.y * (T / 32), red[1] + threadIdx.y * (T / 32)};
    uint4 w[V], xv[V], rv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * T;
        w[i] = c < chunks ? __ldg(reinterpret_cast<const uint4 *>(a.weight) + c) : make_uint4(0, 0, 0, 0);
    }
    auto load = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            const bool in = row < a.N && c < chunks;
            const size_t at = (size_t)row * a.H + c * 8;
            xv[i] = in ? *reinterpret_cast<const uint4 *>(a.x + at) : make_uint4(0, 0, 0, 0);
            if (a.residual) rv[i] = in ? *reinterpret_cast<const uint4 *>(a.residual + at) : make_uint4(0, 0, 0, 0);
        }
    };
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int64_t row0 = (int64_t)blockIdx.x * blockDim.y;  // of the block: every thread makes the same turns
    load(row0 + threadIdx.y);
    for (int b = 0; row0 < a.N; row0 += step, b ^= 1) {
        const int64_t row = row0 + threadIdx.y;
        const size_t at0 = (size_t)row * a.H;
        uint4 s[V];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float f[8];
            s[i] = xv[i];
            unpack8(s[i], f);
            if (a.residual) {
                float r[8];
                unpack8(rv[i], r);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] += r[j];
                s[i] = pack8(f);
                unpack8(s[i], f);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
        }
        load(row + step);
        if (a.residual) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = threadIdx.x + i * T;
                if (row < a.N && c < chunks) *reinterpret_cast<uint4 *>(a.res + at0 + c * 8) = s[i];
            }
        }
        const float inv = 1.0f / sqrtf(row_sum(ss, my_red[b]) / (float)a.H + a.eps);
        if (a.inv_rms && threadIdx.x == 0 && row < a.N) a.inv_rms[row] = inv;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            const bool in = row < a.N && c < chunks;
            float f[8], g[8], y[8];
            unpack8(s[i], f);
            unpack8(w[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = f[j] * g[j] * inv;
            if (a.y && in) *reinterpret_cast<uint4 *>(a.y + at0 + c * 8) = pack8(y);
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
                    *reinterpret_cast<uint2 *>(a.y8 + at0 + c * 8) =
                        make_uint2(pack_e4m3x4(y[0] * is, y[1] * is, y[2] * is, y[3] * is),
                                   pack_e4m3x4(y[4] * is, y[5] * is, y[6] * is, y[7] * is));
                    if ((c & 15) == 0) a.y8_scale[(size_t)row * blocks + (c >> 4)] = (uint8_t)e;
                }
            }
        }
    }
}

// The same walk over the rows; each block sums its rows' dw in registers, adds up
// its row groups and leaves part[block].
template <int V>
__global__ void __launch_bounds__(kNMaxT) add_rmsnorm_bwd_kernel(const NormBwdArgs a) {
    extern __shared__ float sums[];  // [blockDim.y - 1][H] at the end
    __shared__ float red[2][kNMaxT / 32];
    pdl_launch_dependents();
    const int T = blockDim.x, chunks = a.H / 8;
    float *my_red[2] = {red[0] + threadIdx.y * (T / 32), red[1] + threadIdx.y * (T / 32)};
    float dw[V][8];
    uint4 w[V], dv[V], sv[V], gv[V];
    float ninv = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * T;
        w[i] = c < chunks ? __ldg(reinterpret_cast<const uint4 *>(a.weight) + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    }
    auto load = [&](int64_t row) {
        ninv = row < a.N ? __ldg(a.inv_rms + row) : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            const bool in = row < a.N && c < chunks;
            const size_t at = (size_t)row * a.H + c * 8;
            dv[i] = in ? *reinterpret_cast<const uint4 *>(a.dy + at) : make_uint4(0, 0, 0, 0);
            sv[i] = in ? __ldg(reinterpret_cast<const uint4 *>(a.res + at)) : make_uint4(0, 0, 0, 0);
            if (a.dres) gv[i] = in ? *reinterpret_cast<const uint4 *>(a.dres + at) : make_uint4(0, 0, 0, 0);
        }
    };
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int64_t row0 = (int64_t)blockIdx.x * blockDim.y;
    load(row0 + threadIdx.y);
    for (int b = 0; row0 < a.N; row0 += step, b ^= 1) {
        const int64_t row = row0 + threadIdx.y;
        const float inv = ninv;
        uint4 d[V], s[V], g[V];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            d[i] = dv[i], s[i] = sv[i];
            if (a.dres) g[i] = gv[i];
            float fd[8], fs[8], fw[8];
            unpack8(d[i], fd);
            unpack8(s[i], fs);
            unpack8(w[i], fw);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[i][j] = fmaf(fd[j] * inv, fs[j], dw[i][j]);
                dot = fmaf(fd[j] * fw[j], fs[j], dot);
            }
        }
        load(row + step);
        const float k = inv * inv * (row_sum(dot, my_red[b]) / (float)a.H);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            if (row < a.N && c < chunks) {
                float fd[8], fs[8], fw[8], o[8] = {};
                unpack8(d[i], fd);
                unpack8(s[i], fs);
                unpack8(w[i], fw);
                if (a.dres) unpack8(g[i], o);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] += inv * (fd[j] * fw[j] - fs[j] * k);
                *reinterpret_cast<uint4 *>(a.dx + (size_t)row * a.H + c * 8) = pack8(o);
            }
        }
    }
    if (blockDim.y > 1) {
        if (threadIdx.y > 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = threadIdx.x + i * T;
                if (c < chunks)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sums[(threadIdx.y - 1) * a.H + c * 8 + j] = dw[i][j];
            }
        }
        __syncthreads();
        if (threadIdx.y > 0) return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * T;
        if (c < chunks) {
            for (int y = 1; y < (int)blockDim.y; ++y)
#pragma unroll
                for (int j = 0; j < 8; ++j) dw[i][j] += sums[(y - 1) * a.H + c * 8 + j];
            float4 *p = reinterpret_cast<float4 *>(a.part + (size_t)blockIdx.x * a.H + c * 8);
            p[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            p[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    }
}

// dweight[c] = the sum of part[0..parts)[c]: 32 interleaved sums in order, then a
// tree over them.
__global__ void __launch_bounds__(1024) norm_dweight_kernel(const float *part, int parts, int H, float *dweight) {
    __shared__ float sm[32][33];
    const int x = threadIdx.x & 31, g = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    pdl_wait();
    float v = 0.f;
    if (c < H) {
#pragma unroll 4
        for (int i = g; i < parts; i += 32) v += part[(size_t)i * H + c];
    }
    sm[g][x] = v;
    __syncthreads();
    // warp g now adds up column g of the 32
    v = sm[x][g];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (x == 0 && blockIdx.x * 32 + g < H) dweight[blockIdx.x * 32 + g] = v;
}

// Threads per row and chunks per thread: two chunks each where the row has more
// than one warp's worth (one each kept too little in flight: 16384 x 2048 rows took
// 48 us against NNN), four past 8192 columns; short rows share a block of about 256
// threads.
struct NormShape {
    int V, T, R;
};
NormShape norm_shape(int H) {
    const int chunks = H / 8;
    NormShape s;
    s.V = chunks <= 32 ? 1 : chunks <= 2 * kNMaxT ? 2 : 4;
    const int per = (chunks + s.V - 1) / s.V;
    s.T = per <= 16 ? 16 : (per + 31) / 32 * 32;
    s.R = s.T >= 256 ? 1 : 256 / s.T;
    return s;
}
constexpr int kSMThreads = 2048;
#ifndef BWDB
#define BWDB 296
#endif
constexpr int kBwdBlocks = BWDB;

}  // namespace

int norm_bwd_parts(int64_t N, int H) {
    const int64_t groups = (N + norm_shape(H).R - 1) / norm_shape(H).R;
    return (int)(groups < 1 ? 1 : groups < kBwdBlocks ? groups : kBwdBlocks);
}

cudaError_t launch_add_rmsnorm(const NormArgs &a, int num_sms, cudaStream_t s) {
    if (a.N == 0) return cudaSuccess;
    const NormShape n = norm_shape(a.H);
    const int64_t groups = (a.N + n.R - 1) / n.R, room = (int64_t)num_sms * (kSMThreads / (n.T * n.R));
    const dim3 grid((unsigned)(groups < room ? groups : room)), block(n.T, n.R);
    if (n.V == 1) add_rmsnorm_kernel<1><<<grid, block, 0, s>>>(a);
    else if (n.V == 2) add_rmsnorm_kernel<2><<<grid, block, 0, s>>>(a);
    else add_rmsnorm_kernel<4><<<grid, block, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_add_rmsnorm_backward(const NormBwdArgs &a, cudaStream_t s) {
    const NormShape n = norm_shape(a.H);
    const int parts = norm_bwd_parts(a.N, a.H);
    const dim3 block(n.T, n.R);
    const size_t smem = (size_t)(n.R - 1) * a.H * sizeof(float);  // rows of at most 255 * 8 columns share a block: < 17 KB
    if (n.V == 1) add_rmsnorm_bwd_kernel<1><<<parts, block, smem, s>>>(a);
    else if (n.V == 2) add_rmsnorm_bwd_kernel<2><<<parts, block, smem, s>>>(a);
    else add_rmsnorm_bwd_kernel<4><<<parts, block, smem, s>>>(a);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    return launch_maybe_pdl(norm_dweight_kernel, dim3((a.H + 31) / 32), dim3(1024), 0, s, true, (const float *)a.part,
                            parts, a.H, a.dweight);
}

}  // namespace moe
