// 8-bit floating point (e4m3) shared by the norm, the quantisers and the
// block-scaled products: the scale of a block of 128 values, the rounding to
// e4m3, and the launch descriptions.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kScaleBlock = 128;  // values along K per scale (rows); 128 x 128 of a weight
inline int scale_blocks(int64_t n) { return (int)((n + kScaleBlock - 1) / kScaleBlock); }

// What the epilogue of a block-scaled product writes.
// In the forward the products may start as programmatic dependents: the product up
// (SwiGlu) waits for the metadata before it reads any of it and only then lets the
// product down (Y16) start, so that one may read the offsets and load weights at
// once and waits for the product up where it reads h and its scales.  A product on its
// own (Bf16) waits before it reads anything: what starts early is its set-up.
enum Fp8Mode : int32_t {
    kFp8Bf16 = 0,    // out [P,N] bf16
    kFp8SwiGlu = 1,  // h = silu(gate) up as e4m3 [P,N/2] with an e8m0 scale per 128 columns
    // y [P,N] as fp16 scaled by a power of two per 32 columns (the combine's rows, as the bf16 forward's): half
    // the bytes of fp32, which the combine is bound by (95 us for 131072 x 2048), at 2^-11 of a value.  The
    // layer's error against 64 bits goes from 1.664e-3 of its norm, nearly all of it the bf16 output's
    // rounding, to 1.677e-3 (2048 tokens, H 2048, I 768, 128 experts, top 8).
    kFp8Y16 = 2,
};

struct Fp8GemmArgs {
    const uint8_t *w;           // weights [E, N, K] e4m3
    CUtensorMap tmap_w;         // `w` as (K, N rows, E), box 128 x 128 x 1 (made by the launch)
    CUtensorMap tmap_a;         // `a` as (K, rows), box 128 x one chunk (made by the launch; unused when gathered)
    CUtensorMap tmap_out;       // pair kernel: `out` as [P][N] 16-bit, box 32 columns x 32 rows (made by the launch)
    const uint8_t *a;           // rows [rows, K] e4m3
    const void *a_scale;        // [rows, nk]
    const void *w_scale;        // [E, ceil(N/128), nk]
    int32_t a_f32, w_f32;       // scales are fp32 (else e8m0)
    const int32_t *gather;      // [P] row of `a` for sorted position p, or null: p itself
    const int32_t *expert_off;  // [E+1] segment offsets, or null: one segment of P rows
    const __nv_bfloat16 *bias;  // [E,N] or null
    void *out;                  // bf16 [P,N] / e4m3 [P,N/2] / fp16 bits [P,N]
    void *out_scale;            // SwiGlu: e8m0 [P, N/256]; Y16: int8 [P, N/32]
    const WsHeader *hdr;        // skip everything when the metadata aborted, or null
    uint32_t *err;              // device error word, or null
    int64_t P;                  // rows of the output
    int64_t rows;               // rows of `a`
    int32_t E, K, N;
    int32_t nk;                 // ceil(K / 128)
    int32_t layout;             // SwiGlu: MOE_LAYOUT_*
    int32_t split;              // CTAs (few-row kernels) or pairs that share a unit's (tile's) K (set by the launch)
    int32_t pdl;                // launched as a programmatic dependent of the launch before it
};

// Sizes the kernels count in 32 bits and the tensor maps can hold.
inline bool fp8_sizes_ok(int64_t P, int32_t E, int32_t K, int32_t N) {
    const int64_t units = (P / 32 + (E < P ? E : P) + 1) * ((N + 127) / 128);
    return units < INT32_MAX / 2 && (int64_t)K * N < ((int64_t)1 << 39);
}
cudaError_t launch_fp8_gemm(int mode, Fp8GemmArgs &a, int num_sms, cudaStream_t s);       // picks the kernel
// The kernel picked: chunks of so many rows (0: pairs), and how many CTAs (pairs) share a unit's (tile's) K.  fit:
// how many clusters of 2, 4 and 8 CTAs run at once, a byte each (fp8_clusters: on the current device).
struct Fp8Plan {
    int chunk, split;
};
Fp8Plan fp8_plan(int mode, const Fp8GemmArgs &a, int num_sms, int fit);
cudaError_t fp8_clusters(int *fit);
// few rows, e8m0; chunk: 32 or 64 rows, or 128 of one segment
cudaError_t launch_fp8_few_gemm(int mode, Fp8GemmArgs &a, int chunk, int num_sms, cudaStream_t s);
cudaError_t launch_fp8_pair_gemm(int mode, Fp8GemmArgs &a, int num_sms, cudaStream_t s);     // 256-row tiles, any scales
cudaError_t launch_fp8_mx_pair_gemm(int mode, Fp8GemmArgs &a, int num_sms, cudaStream_t s);  // 256-row tiles, e8m0

struct NormArgs {
    const __nv_bfloat16 *x, *residual, *weight;
    __nv_bfloat16 *res, *y;
    uint8_t *y8, *y8_scale;
    float *inv_rms;
    int64_t N;
    int32_t H;
    float eps;
};
cudaError_t launch_add_rmsnorm(const NormArgs &a, int num_sms, cudaStream_t s);
cudaError_t launch_add_rmsnorm_selftest(const NormArgs &a, cudaStream_t s);  // H <= 256, with a residual

struct NormBwdArgs {
    const __nv_bfloat16 *dy, *res, *weight, *dres;
    const float *inv_rms;
    __nv_bfloat16 *dx;
    float *dweight;
    float *part;  // [norm_bwd_parts(N, H), H]
    int64_t N;
    int32_t H;
};
int norm_bwd_parts(int64_t N, int H);
cudaError_t launch_add_rmsnorm_backward(const NormBwdArgs &a, cudaStream_t s);

cudaError_t launch_quantize_rows(const __nv_bfloat16 *x, int64_t M, int32_t K, uint8_t *q, uint8_t *scale,
                                 cudaStream_t s);
cudaError_t launch_quantize_weight(const __nv_bfloat16 *w, int32_t E, int32_t K, int32_t N, uint8_t *q,
                                   uint8_t *scale, cudaStream_t s);

// Host helpers defined in capi.cu.
int current_device_sms(int *sms);  // MOE_OK and the SM count, or the status to return
// e4m3 tensor map: dims/strides/box innermost first, 128-byte swizzle, zero fill.
bool make_map_u8(CUtensorMap *m, const void *ptr, int rank, const uint64_t *dims, const uint64_t *strides,
                 const uint32_t *box);
// 16-bit [rows][cols] tensor map for stores of 32 x 32 boxes, 64-byte swizzle.
bool make_map_out16(CUtensorMap *m, const void *ptr, uint64_t cols, uint64_t rows);

#if defined(__CUDACC__)

// Biased exponent (the e8m0 byte) of a block's scale: the smallest power of two
// s with amax <= 448 s.  448 = 1.75 * 2^8, so s = 2^(e-8) for amax = m 2^e with
// m <= 1.75 and 2^(e-7) above: adding 0x1FFFFF to the mantissa carries into the
// exponent exactly when m > 1.75 (mantissa bits above 0x600000).  1 for a block
// of zeros; at least 2^-126, so that 2^-e is a normal float as well.
__device__ __forceinline__ uint32_t e4m3_scale_exp(float amax) {
    const uint32_t b = __float_as_uint(amax);
    if (b == 0) return 127u;
    return (uint32_t)max((int)((b + 0x1FFFFFu) >> 23) - 8, 1);
}
__device__ __forceinline__ float scale_of_exp(uint32_t e) { return __uint_as_float(e << 23); }          // 1..254
__device__ __forceinline__ float inv_scale_of_exp(uint32_t e) { return __uint_as_float((254u - e) << 23); }  // 1..253

// A load of what a launch before may have written: it stays behind the wait for that launch, which this
// one overlaps (pdl_wait).  The read-only loads (__ldg) take memory that nobody writes while the kernel
// runs, and the compiler may move them ahead of the wait.  Nothing waits for it here.
template <typename T>
__device__ __forceinline__ T load_now(const T *p) {
    static_assert(sizeof(T) == 4, "a 32-bit word");
    T v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t load_now(const uint8_t *p) {
    uint32_t v;
    asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// A scale in two steps, for loads that should be in flight together: the raw bits of
// n scales (e8m0 bytes or fp32) from index i on (behind `last` more, the last one
// repeated), and their values (e8m0: 0 is 2^-127, 255 is NaN).
template <int n>
__device__ __forceinline__ void load_scale_bits(const void *p, int f32, size_t i, int last, uint32_t (&raw)[n]) {
    if (f32) {
#pragma unroll
        for (int k = 0; k < n; ++k) raw[k] = load_now(static_cast<const uint32_t *>(p) + i + min(k, last));
    } else {
#pragma unroll
        for (int k = 0; k < n; ++k) raw[k] = load_now(static_cast<const uint8_t *>(p) + i + min(k, last));
    }
}
__device__ __forceinline__ float scale_of_bits(uint32_t raw, int f32) {
    return __uint_as_float(f32 ? raw : raw == 0 ? 0x00400000u : raw == 255u ? 0x7FC00000u : raw << 23);
}

// Infinities become NaN (e4m3 has no infinity, and the conversion would
// saturate them); every other value is unchanged.
__device__ __forceinline__ float inf_to_nan(float v) { return fmaf(v, 0.0f, v); }
// |v| for a block's maximum: 0 for NaN (fmaxf drops NaN).
__device__ __forceinline__ float amax_of(float m, float v) { return fmaxf(m, fabsf(v)); }

// Two values, already divided by the scale, rounded to nearest even: lo in bits 0-7.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    return pack_e4m3x2(a, b) | (pack_e4m3x2(c, d) << 16);
}

// D[tmem] (+)= A[smem desc] * B[smem desc], kind::f8f6f4 (e4m3 in, fp32 accumulate), K = 32.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor, kind::f8f6f4: fp32 accumulate, A and B e4m3 (format 0), both K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | ((static_cast<uint32_t>(N) >> 3) << 17) | ((static_cast<uint32_t>(M) >> 4) << 24);
}

// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

#endif  // __CUDACC__

}  // namespace moe
