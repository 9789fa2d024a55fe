// What the kernels share that let the tensor cores apply e8m0 scales
// (tcgen05.mma.kind::mxf8f6f4.block_scale).
#pragma once

#include "fp8_pair.cuh"

namespace moe {

#if defined(__CUDACC__)

// Instruction descriptor, kind::mxf8f6f4: A and B e4m3 (format 0), both K-major, e8m0 scales
// (bit 23), M x N; idesc_byte(k) adds the byte of the scale words to use (bits 4-5 for B,
// 29-30 for A).
__host__ __device__ constexpr uint32_t idesc_mx_e4m3(int M, int N) {
    return ((static_cast<uint32_t>(N) >> 3) << 17) | (1u << 23) | ((static_cast<uint32_t>(M) >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_byte(int k) { return (uint32_t)k << 4 | (uint32_t)k << 29; }
// 32 lanes x 4 (8) 32-bit TMEM columns from registers.
__device__ __forceinline__ void tmem_st_x4(uint32_t taddr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r0), "r"(r1),
                 "r"(r2), "r"(r3)
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The e8m0 bytes i .. i + 3 of a row of scales, as two registers that make up one
// word by r0 | r1 << 16 -- later: nothing here waits for the loads, except where a
// row starts at an odd byte.  how: 0 rows of whole words, 1 of half-words, 2 bytes.
__device__ __forceinline__ void load_e8m0_x4(const uint8_t *p, size_t i, int last, int how, uint32_t &r0, uint32_t &r1) {
    const uint8_t *q = p + i;
    r1 = 0;
    if (how == 0) {
        r0 = __ldg(reinterpret_cast<const uint32_t *>(q));
    } else if (how == 1) {
        r0 = __ldg(reinterpret_cast<const uint16_t *>(q));
        if (last >= 2) r1 = __ldg(reinterpret_cast<const uint16_t *>(q + 2));
    } else {  // behind `last` the last byte again: never used
        const uint32_t b0 = __ldg(q), b1 = __ldg(q + min(1, last)), b2 = __ldg(q + min(2, last)),
                       b3 = __ldg(q + min(3, last));
        r0 = b0 | b1 << 8 | b2 << 16 | b3 << 24;
    }
}
__device__ __forceinline__ int e8m0_rows(const uint8_t *p, int nk) {
    const uint32_t a = (uint32_t)reinterpret_cast<uintptr_t>(p) | (uint32_t)nk;
    return (a & 3) == 0 ? 0 : (a & 1) == 0 ? 1 : 2;
}

#endif  // __CUDACC__

}  // namespace moe
