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
//
// Bound by HBM: one pass, every tensor read or written once.  Every kernel is a
// programmatic dependent of the launch before it: its blocks come up and set their
// barriers while that one ends.  Measured back to back in a graph (rates of the bytes that have
// to move): 16384 x 2048 with residual, 8-bit out 42 us (5.7 TB/s; 45 without the early
// start); 8191 x 7168 with residual, bf16 out 77 us (6.1 TB/s; 79); gradient of 16384
// x 2048 with dres 47 us (5.7 TB/s; 49), its second kernel included.  Without a
// residual the 8-bit form has half as many bytes to an instruction and issues most of the
// time: 16384 x 2048 29 us (3.5 TB/s; 32 with two products per value and IEEE divisions), 65536 x 2048
// 109 us with 21 instructions a value, polling included, the schedulers busy 74 % of the cycles and
// DRAM 42 %.
#include "fp8.cuh"

namespace moe {
namespace {

constexpr int kNMaxT = 512;  // threads per row at most
constexpr float kLargest = 3.402823466e38f;
constexpr int kStages = 2;   // of the ring (four: 16384 x 2048 55 us against 43, 8191 x 7168 80 against 75)

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    f[0] = bf16lo(v.x), f[1] = bf16hi(v.x), f[2] = bf16lo(v.y), f[3] = bf16hi(v.y);
    f[4] = bf16lo(v.z), f[5] = bf16hi(v.z), f[6] = bf16lo(v.w), f[7] = bf16hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// Sum over the T threads of one row (T = blockDim.x: 16, or a multiple of 32), the
// same value in each, behind a barrier of the whole block.  red: this row's T / 32
// floats; a caller that comes again passes another buffer in between.
__device__ __forceinline__ float row_sum(float v, float *red) {
    const int T = blockDim.x;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (T > 16) v += __shfl_xor_sync(0xffffffffu, v, 16);
    if (T > 32 && (threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    if (T <= 32) return v;
    float t = 0.f;
    for (int i = 0; i < T / 32; ++i) t += red[i];
    return t;
}

// A block's rows on their way in: a ring of stages, each blockDim.y neighbouring rows
// of kIn tensors (whole rows are contiguous: one bulk copy per tensor), loaded ahead
// by thread (0, 0).  What the loads need in flight -- several times what two loads per
// thread can hold -- then costs shared memory instead of registers.
// kLose (self-test): the loads from the block's third turn on never come, and waits give up after 20 ms.
template <int kIn, bool kLose = false>
struct RowRing {
    const __nv_bfloat16 *src[kIn];
    uint32_t bars, data;  // shared addresses: a barrier per stage, the stages
    uint32_t row_bytes, stage_bytes;
    int64_t N, step;
    bool leader;
    uint32_t *gave_up;

    __device__ __forceinline__ void start(uint32_t smem, int H, int64_t n, int64_t first, uint32_t *flag) {
        bars = smem;
        data = smem + 64;
        row_bytes = (uint32_t)H * 2;
        stage_bytes = row_bytes * blockDim.y;
        N = n;
        step = (int64_t)gridDim.x * blockDim.y;
        leader = threadIdx.x == 0 && threadIdx.y == 0;
        gave_up = flag;
        if (leader) {
            *flag = 0;
            for (int s = 0; s < kStages; ++s) mbar_init(bars + 8 * s, 1);
            fence_barrier_init();
        }
        __syncthreads();
        pdl_wait();  // nothing is read or written before
        pdl_launch_dependents();
        if (leader)
            for (int s = 0; s < kStages; ++s) fetch(s, first + s * step);
    }
    __device__ __forceinline__ uint32_t at(int stage, int t) const { return data + (stage * kIn + t) * stage_bytes; }
    // thread (0, 0): load the block's rows from row0 on into a stage that nobody reads any more
    __device__ __forceinline__ void fetch(int stage, int64_t row0) const {
        if (row0 >= N || *(volatile uint32_t *)gave_up) return;
        if (kLose && row0 >= 2 * step) return;
        const int64_t left = N - row0;
        const uint32_t bytes = row_bytes * (uint32_t)(left < blockDim.y ? left : blockDim.y);
        mbar_arrive_expect_tx(bars + 8 * stage, kIn * bytes);
#pragma unroll
        for (int t = 0; t < kIn; ++t)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             at(stage, t)),
                         "l"(reinterpret_cast<const char *>(src[t]) + (size_t)row0 * row_bytes), "r"(bytes),
                         "r"(bars + 8 * stage)
                         : "memory");
    }
    __device__ __forceinline__ void wait(int stage, uint32_t phase) const {
        mbar_wait_bounded(bars + 8 * stage, phase, gave_up, kLose ? 20000000ull : kWaitTimeoutNs);
    }
    // behind the last row; after a wait that gave up: time for copies in flight to land
    __device__ __forceinline__ void end() const {
        if (!*(volatile uint32_t *)gave_up) return;
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
    }
    __device__ __forceinline__ uint4 chunk(int stage, int t, int c) const {
        uint4 v;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(at(stage, t) + threadIdx.y * row_bytes + (uint32_t)c * 16)
                     : "memory");
        return v;
    }
};

// This thread's chunks of a row: NaN.
__device__ __noinline__ void nan_row(__nv_bfloat16 *row, int chunks) {
    for (int c = threadIdx.x; c < chunks; c += blockDim.x)
        *reinterpret_cast<uint4 *>(row + c * 8) = make_uint4(~0u, ~0u, ~0u, ~0u);
}

// Thread (x, y) of a block works on row y of the block's rows, on the 8-column
// chunks x, x + T, ... (V of them); a block takes rows until there are none.
template <int V, bool kResidual, bool kLose = false>
__global__ void __launch_bounds__(kNMaxT, 2) add_rmsnorm_kernel(const NormArgs a) {
    extern __shared__ __align__(128) uint8_t ring_smem[];
    __shared__ float red[2][kNMaxT / 32];
    __shared__ uint32_t gave_up;
    const int T = blockDim.x, chunks = a.H / 8;
    const float per_h = 1.0f / (float)a.H;
    const int blocks = (a.H + kScaleBlock - 1) / kScaleBlock;
    float *my_red[2] = {red[0] + threadIdx.y * (T / 32), red[1] + threadIdx.y * (T / 32)};
    int64_t row0 = (int64_t)blockIdx.x * blockDim.y;  // of the block: every thread makes the same turns
    RowRing<kResidual ? 2 : 1, kLose> ring;
    ring.src[0] = a.x;
    if (kResidual) ring.src[kResidual ? 1 : 0] = a.residual;
    ring.start(smem_u32(ring_smem), a.H, a.N, row0, &gave_up);
    uint4 w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * T;
        w[i] = c < chunks ? reinterpret_cast<const uint4 *>(a.weight)[c] : make_uint4(0, 0, 0, 0);
    }
    int stage = 0;
    uint32_t phase = 0;
    int64_t lost = -1;  // this thread's first row whose load did not come
    for (int b = 0; row0 < a.N; row0 += ring.step, b ^= 1) {
        const int64_t row = row0 + threadIdx.y;
        const size_t at0 = (size_t)row * a.H;
        ring.wait(stage, phase);
        uint4 s[V];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            const bool in = row < a.N && c < chunks;
            s[i] = in ? ring.chunk(stage, 0, c) : make_uint4(0, 0, 0, 0);
            float f[8];
            unpack8(s[i], f);
            if (kResidual && in) {
                float r[8];
                unpack8(ring.chunk(stage, kResidual ? 1 : 0, c), r);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] += r[j];
                s[i] = pack8(f);
                unpack8(s[i], f);
                *reinterpret_cast<uint4 *>(a.res + at0 + c * 8) = s[i];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
        }
        ss = row_sum(ss, my_red[b]);  // and every thread has read the stage
        if (ring.leader) ring.fetch(stage, row0 + kStages * ring.step);
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
        }
        float inv = rsqrtf(fmaf(ss, per_h, a.eps));  // (within 2 units in the last place)
        if (*(volatile uint32_t *)&gave_up) {  // a load never came: NaN, not a wrong value
            inv = __uint_as_float(0x7FC00000u);
            if (lost < 0) lost = row;
        }
        if (a.inv_rms && threadIdx.x == 0 && row < a.N) a.inv_rms[row] = inv;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            const bool in = row < a.N && c < chunks;
            float f[8], g[8], v[8];
            unpack8(s[i], f);
            unpack8(w[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = f[j] * g[j];
            if (a.y && in) {
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = v[j] * inv;
                *reinterpret_cast<uint4 *>(a.y + at0 + c * 8) = pack8(y);
            }
            if (a.y8) {
                // 16 consecutive threads hold one block of 128 columns.  Its largest |y| is the largest
                // |s w| times inv (rounding keeps the order), and inv / scale is exact, so that a value
                // costs one product and the conversion.
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = amax_of(m, v[j]);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                m *= inv;
                uint32_t e = e4m3_scale_exp(m);
                float k = inv * inv_scale_of_exp(min(e, 253u));
                if (__any_sync(0xffffffffu, !(fmaxf(m, k) <= kLargest) || m != m)) {
                    // an infinity or a NaN among them, or inv / scale past the range: value by value
                    m = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        v[j] = inf_to_nan(v[j] * inv);
                        m = amax_of(m, v[j]);
                    }
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    e = e4m3_scale_exp(m);
                    k = inv_scale_of_exp(e);
                }
                if (in) {
                    *reinterpret_cast<uint2 *>(a.y8 + at0 + c * 8) =
                        make_uint2(pack_e4m3x4(v[0] * k, v[1] * k, v[2] * k, v[3] * k),
                                   pack_e4m3x4(v[4] * k, v[5] * k, v[6] * k, v[7] * k));
                    if ((c & 15) == 0) a.y8_scale[(size_t)row * blocks + (c >> 4)] = (uint8_t)e;
                }
            }
        }
    }
    ring.end();
    // s has been written from whatever was there (at the row itself this cost a single row 0.1 us)
    if (kResidual && lost >= 0)
        for (; lost < a.N; lost += ring.step) nan_row(a.res + (size_t)lost * a.H, chunks);
}

// The same walk over the rows; each block sums its rows' dw in registers, adds up
// its row groups and leaves part[block].
template <int V, bool kDres>
__global__ void __launch_bounds__(kNMaxT) add_rmsnorm_bwd_kernel(const NormBwdArgs a) {
    extern __shared__ __align__(128) uint8_t ring_smem[];  // at the end [blockDim.y - 1][H] sums
    __shared__ float red[2][kNMaxT / 32];
    __shared__ uint32_t gave_up;
    const int T = blockDim.x, chunks = a.H / 8;
    const float per_h = 1.0f / (float)a.H;
    float *my_red[2] = {red[0] + threadIdx.y * (T / 32), red[1] + threadIdx.y * (T / 32)};
    int64_t row0 = (int64_t)blockIdx.x * blockDim.y;
    RowRing<kDres ? 3 : 2> ring;
    ring.src[0] = a.dy;
    ring.src[1] = a.res;
    if (kDres) ring.src[kDres ? 2 : 0] = a.dres;
    ring.start(smem_u32(ring_smem), a.H, a.N, row0, &gave_up);
    float dw[V][8];
    uint4 w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * T;
        w[i] = c < chunks ? reinterpret_cast<const uint4 *>(a.weight)[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    }
    int stage = 0;
    uint32_t phase = 0;
    for (int b = 0; row0 < a.N; row0 += ring.step, b ^= 1) {
        const int64_t row = row0 + threadIdx.y;
        const float inv = row < a.N ? a.inv_rms[row] : 0.f;
        ring.wait(stage, phase);
        uint4 d[V], s[V], g[V];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            const bool in = row < a.N && c < chunks;
            d[i] = in ? ring.chunk(stage, 0, c) : make_uint4(0, 0, 0, 0);
            s[i] = in ? ring.chunk(stage, 1, c) : make_uint4(0, 0, 0, 0);
            if (kDres) g[i] = in ? ring.chunk(stage, kDres ? 2 : 0, c) : make_uint4(0, 0, 0, 0);
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
        dot = row_sum(dot, my_red[b]);  // and every thread has read the stage
        if (ring.leader) ring.fetch(stage, row0 + kStages * ring.step);
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
        }
        if (*(volatile uint32_t *)&gave_up) dot = __uint_as_float(0x7FC00000u);  // a load never came: NaN, not a wrong value
        const float k = inv * (inv * (dot * per_h));  // (inv^2 alone may pass the range)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            if (row < a.N && c < chunks) {
                float fd[8], fs[8], fw[8], o[8] = {};
                unpack8(d[i], fd);
                unpack8(s[i], fs);
                unpack8(w[i], fw);
                if (kDres) unpack8(g[i], o);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] += inv * (fd[j] * fw[j] - fs[j] * k);
                *reinterpret_cast<uint4 *>(a.dx + (size_t)row * a.H + c * 8) = pack8(o);
            }
        }
    }
    ring.end();
    // (a ring that gave up: dweight NaN as well)
    const float bad = *(volatile uint32_t *)&gave_up ? __uint_as_float(0x7FC00000u) : 0.f;
    if (blockDim.y > 1) {
        float *sums = reinterpret_cast<float *>(ring_smem + 64);
        __syncthreads();  // (no load is in flight: every fetch has been waited for)
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
            for (int y = 1; y < (int)blockDim.y; ++y) {
                const float *sums = reinterpret_cast<const float *>(ring_smem + 64);
#pragma unroll
                for (int j = 0; j < 8; ++j) dw[i][j] += sums[(y - 1) * a.H + c * 8 + j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) dw[i][j] += bad;
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
    pdl_launch_dependents();
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

// Threads per row and chunks per thread: two chunks each where the row has more than
// one warp's worth, four past 8192 columns; short rows share a block of about 256
// threads.
struct NormShape {
    int V, T, R;
    size_t smem(int H, int tensors) const {
        const size_t ring = 64 + (size_t)kStages * R * H * 2 * tensors;
        const size_t sums = 64 + (size_t)(R - 1) * H * 4;  // the gradient's row groups, in the ring's place
        return ring > sums ? ring : sums;
    }
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
constexpr int kBwdBlocks = 296;  // two on each of 148 SMs (148: 64 us for 16384 x 2048 against 49; 592: 54)

template <typename Kernel, typename Args>
cudaError_t launch_rows(Kernel kernel, const Args &a, const NormShape &n, int tensors, unsigned grid, cudaStream_t s) {
    int unused = 0;
    const cudaError_t err = launch_setup_once((const void *)kernel, &unused, [&](int, int *v) -> cudaError_t {
        *v = 1;
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 << 10);
    });
    if (err != cudaSuccess) return err;
    return launch_maybe_pdl(kernel, dim3(grid), dim3(n.T, n.R), n.smem(a.H, tensors), s, true, a);
}
template <bool kResidual>
cudaError_t launch_forward(const NormArgs &a, int num_sms, cudaStream_t s) {
    const NormShape n = norm_shape(a.H);
    // Four blocks to an SM stay resident.  Where a bf16 y is written as well, more waves of blocks,
    // which stagger loads and stores, are faster on long rows: eight to an SM (16384 x 2048 with
    // residual 45.9 us against 48.6, 8191 x 7168 76 against 81), or three row groups to a block
    // where s is written too, rows are many and no wider than 4096 (40000 x 2048 101 against 111,
    // 16384 x 2048 44.6 against 45.3; 8191 x 7168 79.3 against 76.8).  Not on short rows (50000 x
    // 256 16.4 against 16.0) nor with y8 alone (8191 x 7168 71.7 against 71.1).
    const int64_t groups = (a.N + n.R - 1) / n.R, four = 4 * (int64_t)num_sms, thirds = (groups + 2) / 3;
    const bool more = a.y && a.H >= 1024 && a.H <= 8192;
    const int64_t room = !more ? four : kResidual && a.H <= 4096 && thirds > 2 * four ? thirds : 2 * four;
    const unsigned grid = (unsigned)(groups < room ? groups : room);
    const int in = kResidual ? 2 : 1;
    if (n.V == 1) return launch_rows(add_rmsnorm_kernel<1, kResidual>, a, n, in, grid, s);
    if (n.V == 2) return launch_rows(add_rmsnorm_kernel<2, kResidual>, a, n, in, grid, s);
    return launch_rows(add_rmsnorm_kernel<4, kResidual>, a, n, in, grid, s);
}
template <bool kDres>
cudaError_t launch_backward(const NormBwdArgs &a, cudaStream_t s) {
    const NormShape n = norm_shape(a.H);
    const unsigned grid = (unsigned)norm_bwd_parts(a.N, a.H);
    const int in = kDres ? 3 : 2;
    if (n.V == 1) return launch_rows(add_rmsnorm_bwd_kernel<1, kDres>, a, n, in, grid, s);
    if (n.V == 2) return launch_rows(add_rmsnorm_bwd_kernel<2, kDres>, a, n, in, grid, s);
    return launch_rows(add_rmsnorm_bwd_kernel<4, kDres>, a, n, in, grid, s);
}

}  // namespace

cudaError_t launch_add_rmsnorm_selftest(const NormArgs &a, cudaStream_t s) {
    return launch_rows(add_rmsnorm_kernel<1, true, true>, a, norm_shape(a.H), 2, 1, s);
}

int norm_bwd_parts(int64_t N, int H) {
    const int64_t groups = (N + norm_shape(H).R - 1) / norm_shape(H).R;
    return (int)(groups < 1 ? 1 : groups < kBwdBlocks ? groups : kBwdBlocks);
}

cudaError_t launch_add_rmsnorm(const NormArgs &a, int num_sms, cudaStream_t s) {
    if (a.N == 0) return cudaSuccess;
    return a.residual ? launch_forward<true>(a, num_sms, s) : launch_forward<false>(a, num_sms, s);
}

cudaError_t launch_add_rmsnorm_backward(const NormBwdArgs &a, cudaStream_t s) {
    const cudaError_t err = a.dres ? launch_backward<true>(a, s) : launch_backward<false>(a, s);
    if (err != cudaSuccess) return err;
    return launch_maybe_pdl(norm_dweight_kernel, dim3((a.H + 31) / 32), dim3(1024), 0, s, true, (const float *)a.part,
                            norm_bwd_parts(a.N, a.H), a.H, a.dweight);
}

}  // namespace moe
