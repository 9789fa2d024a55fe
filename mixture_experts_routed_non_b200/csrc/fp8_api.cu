// C entry points of the norm, the quantisers and the block-scaled products:
// argument checks and one launch each (the forward in 8 bits sits with the
// bf16 forward in capi.cu).
#include <string.h>

#include "fp8.cuh"

using namespace moe;

namespace {

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - (1 << 20);
constexpr int32_t kMaxNormH = 16384;  // columns a block of 512 threads holds, 32 each

bool scale_ok(const void *p, int32_t dtype) {
    return dtype == MOE_SCALE_E8M0 || (dtype == MOE_SCALE_F32 && ptr_aligned(p, 4));
}

int product(const void *a, const void *a_scale, int32_t a_sd, int64_t rows, int32_t K, const int32_t *gather,
            int64_t P, const int32_t *expert_off, int32_t E, const void *w, const void *w_scale, int32_t w_sd,
            int32_t N, const void *bias, void *out, uint32_t *err_word, moe_stream_t stream) {
    if (P < 0 || P >= kMaxRows || rows < 0 || rows >= kMaxRows || E < 1 || E > kMaxExperts) return MOE_ERR_ARG;
    if (K < 16 || K % 16 != 0 || N < 8 || N % 8 != 0 || K > (1 << 28) || N > (1 << 28)) return MOE_ERR_SHAPE;
    if (!fp8_sizes_ok(P, E, K, N)) return MOE_ERR_SHAPE;
    if (!w || !w_scale || (P > 0 && !out) || (rows > 0 && (!a || !a_scale))) return MOE_ERR_ARG;
    if (gather ? !ptr_aligned(gather, 4) : P != rows) return MOE_ERR_ARG;
    if (P > 0 && rows == 0) return MOE_ERR_ARG;
    if (!ptr_aligned(a, 16) || !ptr_aligned(w, 16) || !ptr_aligned(out, 16) || !ptr_aligned(bias, 2) ||
        !ptr_aligned(expert_off, 4) || !ptr_aligned(err_word, 4) || !scale_ok(a_scale, a_sd) ||
        !scale_ok(w_scale, w_sd))
        return MOE_ERR_ARG;
    int sms = 0;
    const int st = current_device_sms(&sms);
    if (st) return st;
    if (P == 0) return MOE_OK;
    Fp8GemmArgs g;
    memset(&g, 0, sizeof g);
    g.w = static_cast<const uint8_t *>(w);
    g.a = static_cast<const uint8_t *>(a);
    g.a_scale = a_scale;
    g.w_scale = w_scale;
    g.a_f32 = a_sd == MOE_SCALE_F32;
    g.w_f32 = w_sd == MOE_SCALE_F32;
    g.gather = gather;
    g.expert_off = expert_off;
    g.bias = static_cast<const __nv_bfloat16 *>(bias);
    g.out = out;
    g.err = err_word;
    g.P = P;
    g.rows = rows;
    g.E = E;
    g.K = K;
    g.N = N;
    g.nk = scale_blocks(K);
    g.pdl = 1;
    return launch_fp8_gemm(kFp8Bf16, g, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                                      : MOE_ERR_CUDA;
}

// The norm's arguments checked (the device last) and put together.
int norm_args(const void *x, const void *residual, const void *weight, int64_t N, int32_t H, float eps, void *res,
              void *y, void *y8, void *y8_scale, float *inv_rms, NormArgs *a, int *sms) {
    if (N < 0 || N >= kMaxRows || !(eps >= 0.f)) return MOE_ERR_ARG;
    if (H < 8 || H % 8 != 0 || H > kMaxNormH) return MOE_ERR_SHAPE;
    if (!weight) return MOE_ERR_ARG;
    // without rows the row buffers may be empty (null)
    if (N > 0 && (!x || (!residual) != (!res) || (!y8) != (!y8_scale) || (!y && !y8))) return MOE_ERR_ARG;
    if (!ptr_aligned(x, 16) || !ptr_aligned(residual, 16) || !ptr_aligned(weight, 16) || !ptr_aligned(res, 16) ||
        !ptr_aligned(y, 16) || !ptr_aligned(y8, 16) || !ptr_aligned(inv_rms, 4))
        return MOE_ERR_ARG;
    const int st = current_device_sms(sms);
    if (st) return st;
    a->x = static_cast<const __nv_bfloat16 *>(x);
    a->residual = static_cast<const __nv_bfloat16 *>(residual);
    a->weight = static_cast<const __nv_bfloat16 *>(weight);
    a->res = static_cast<__nv_bfloat16 *>(res);
    a->y = static_cast<__nv_bfloat16 *>(y);
    a->y8 = static_cast<uint8_t *>(y8);
    a->y8_scale = static_cast<uint8_t *>(y8_scale);
    a->inv_rms = inv_rms;
    a->N = N;
    a->H = H;
    a->eps = eps;
    return MOE_OK;
}

}  // namespace

extern "C" MOE_API int moe_add_rmsnorm(const void *x, const void *residual, const void *weight, int64_t N, int32_t H,
                                       float eps, void *res, void *y, void *y8, void *y8_scale, float *inv_rms,
                                       moe_stream_t stream) {
    NormArgs a;
    int sms = 0;
    const int st = norm_args(x, residual, weight, N, H, eps, res, y, y8, y8_scale, inv_rms, &a, &sms);
    if (st) return st;
    return launch_add_rmsnorm(a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" MOE_API int moe_add_rmsnorm_selftest_wait_timeout(const void *x, const void *residual, const void *weight,
                                                             int64_t N, int32_t H, float eps, void *res, void *y,
                                                             float *inv_rms, moe_stream_t stream) {
    if (N < 1 || N > 4096 || !residual || !y) return MOE_ERR_ARG;  // (every turn behind the lost one polls a while)
    if (H > 256) return MOE_ERR_SHAPE;
    NormArgs a;
    int sms = 0;
    const int st = norm_args(x, residual, weight, N, H, eps, res, y, nullptr, nullptr, inv_rms, &a, &sms);
    if (st) return st;
    return launch_add_rmsnorm_selftest(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" MOE_API size_t moe_add_rmsnorm_backward_workspace_bytes(int64_t N, int32_t H) {
    if (N < 0 || N >= kMaxRows || H < 8 || H % 8 != 0 || H > kMaxNormH) return 0;
    return (size_t)norm_bwd_parts(N, H) * H * sizeof(float);
}

extern "C" MOE_API int moe_add_rmsnorm_backward(const void *dy, const void *res, const void *weight,
                                                const float *inv_rms, const void *dres, int64_t N, int32_t H, void *dx,
                                                float *dweight, void *ws, size_t ws_bytes, moe_stream_t stream) {
    if (N < 0 || N >= kMaxRows) return MOE_ERR_ARG;
    if (H < 8 || H % 8 != 0 || H > kMaxNormH) return MOE_ERR_SHAPE;
    if (!weight || !dweight || (N > 0 && (!dy || !res || !inv_rms || !dx))) return MOE_ERR_ARG;
    if (!ptr_aligned(dy, 16) || !ptr_aligned(res, 16) || !ptr_aligned(weight, 16) || !ptr_aligned(dres, 16) ||
        !ptr_aligned(dx, 16) || !ptr_aligned(inv_rms, 4) || !ptr_aligned(dweight, 4))
        return MOE_ERR_ARG;
    if (!ws || !ptr_aligned(ws, 256) || ws_bytes < moe_add_rmsnorm_backward_workspace_bytes(N, H)) return MOE_ERR_WS;
    int sms = 0;
    const int st = current_device_sms(&sms);
    if (st) return st;
    NormBwdArgs a;
    a.dy = static_cast<const __nv_bfloat16 *>(dy);
    a.res = static_cast<const __nv_bfloat16 *>(res);
    a.weight = static_cast<const __nv_bfloat16 *>(weight);
    a.dres = static_cast<const __nv_bfloat16 *>(dres);
    a.inv_rms = inv_rms;
    a.dx = static_cast<__nv_bfloat16 *>(dx);
    a.dweight = dweight;
    a.part = static_cast<float *>(ws);
    a.N = N;
    a.H = H;
    return launch_add_rmsnorm_backward(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                                   : MOE_ERR_CUDA;
}

extern "C" MOE_API int moe_fp8_quantize_rows(const void *x, int64_t M, int32_t K, void *q, void *scale,
                                             moe_stream_t stream) {
    if (M < 0 || M >= kMaxRows || (M > 0 && (!x || !q || !scale))) return MOE_ERR_ARG;
    if (K < 16 || K % 16 != 0 || K > (1 << 28)) return MOE_ERR_SHAPE;
    if (M * scale_blocks(K) >= (int64_t)1 << 36) return MOE_ERR_SHAPE;  // 64 scale blocks to a block of the launch grid
    if (!ptr_aligned(x, 16) || !ptr_aligned(q, 16)) return MOE_ERR_ARG;
    int sms = 0;
    const int st = current_device_sms(&sms);
    if (st) return st;
    return launch_quantize_rows(static_cast<const __nv_bfloat16 *>(x), M, K, static_cast<uint8_t *>(q),
                                static_cast<uint8_t *>(scale),
                                reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

extern "C" MOE_API int moe_fp8_quantize_weight(const void *w, int32_t E, int32_t K, int32_t N, void *q, void *scale,
                                               moe_stream_t stream) {
    if (E < 1 || E > kMaxExperts || !w || !q || !scale) return MOE_ERR_ARG;
    // one block of the launch grid per 128 rows of N: at most 65535 of them
    if (K < 16 || K % 16 != 0 || K > (1 << 28) || N < 8 || N % 8 != 0 || N > 65535 * kScaleBlock) return MOE_ERR_SHAPE;
    if (!ptr_aligned(w, 16) || !ptr_aligned(q, 16)) return MOE_ERR_ARG;
    int sms = 0;
    const int st = current_device_sms(&sms);
    if (st) return st;
    return launch_quantize_weight(static_cast<const __nv_bfloat16 *>(w), E, K, N, static_cast<uint8_t *>(q),
                                  static_cast<uint8_t *>(scale),
                                  reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

extern "C" MOE_API int moe_fp8_linear(const void *a, const void *a_scale, int32_t a_scale_dtype, int64_t M, int32_t K,
                                      const void *w, const void *w_scale, int32_t w_scale_dtype, int32_t N,
                                      const void *bias, void *out, uint32_t *err_word, moe_stream_t stream) {
    return product(a, a_scale, a_scale_dtype, M, K, nullptr, M, nullptr, 1, w, w_scale, w_scale_dtype, N, bias, out,
                   err_word, stream);
}

extern "C" MOE_API int moe_fp8_grouped_linear(const void *a, const void *a_scale, int32_t a_scale_dtype, int64_t rows,
                                              int32_t K, const int32_t *gather, int64_t P, const int32_t *expert_off,
                                              int32_t E, const void *w, const void *w_scale, int32_t w_scale_dtype,
                                              int32_t N, const void *bias, void *out, uint32_t *err_word,
                                              moe_stream_t stream) {
    if (!expert_off) return MOE_ERR_ARG;
    return product(a, a_scale, a_scale_dtype, rows, K, gather, P, expert_off, E, w, w_scale, w_scale_dtype, N, bias,
                   out, err_word, stream);
}

extern "C" MOE_API int moe_fp8_product_plan(int32_t swiglu, int32_t f32_scales, int64_t P, int32_t K, int32_t N, int32_t E,
                                            int32_t num_sms, const int32_t *clusters, int32_t *chunk, int32_t *split) {
    if (!chunk || !split || P < 1 || P >= kMaxRows || E < 0 || E > kMaxExperts || num_sms < 0) return MOE_ERR_ARG;
    if ((num_sms > 0) != (clusters != nullptr) || (swiglu && E == 0)) return MOE_ERR_ARG;
    if (K < 16 || K % 16 != 0 || N < 8 || N % (swiglu ? 256 : 8) != 0 || K > (1 << 28) || N > (1 << 28)) return MOE_ERR_SHAPE;
    if (!fp8_sizes_ok(P, E ? E : 1, K, N)) return MOE_ERR_SHAPE;
    int sms = num_sms, fit = 0;
    if (!clusters) {
        const int st = current_device_sms(&sms);
        if (st) return st;
        if (fp8_clusters(&fit) != cudaSuccess) return MOE_ERR_CUDA;
    } else {
        for (int i = 0; i < 3; ++i) {
            if (clusters[i] < 0 || clusters[i] > 255) return MOE_ERR_ARG;
            fit |= clusters[i] << (8 * i);
        }
    }
    const int32_t offsets = 0;  // (only whether there are segments matters)
    Fp8GemmArgs g;
    memset(&g, 0, sizeof g);
    g.expert_off = E ? &offsets : nullptr;
    g.a_f32 = g.w_f32 = f32_scales != 0;
    g.P = P;
    g.E = E ? E : 1;
    g.K = K;
    g.N = N;
    g.nk = scale_blocks(K);
    const Fp8Plan p = fp8_plan(swiglu ? kFp8SwiGlu : kFp8Bf16, g, sms, fit);
    *chunk = p.chunk;
    *split = p.split;
    return MOE_OK;
}
