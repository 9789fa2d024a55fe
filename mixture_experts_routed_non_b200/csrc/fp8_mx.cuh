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
// 32 lanes x 4 32-bit TMEM columns from registers.
__device__ __forceinline__ void tmem_st_x4(uint32_t taddr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r0), "r"(r1),
                 "r"(r2), "r"(r3)
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The e8m0 bytes i .. i + 3 of a row of scales, up to `last` of them behind the first, in
// two registers: the aligned words they lie in (the second only where it holds one of
// them), and the shift that brings the first byte to the bottom in the low five bits of the
// next field of `shifts`.  e8m0_word joins them -- later: nothing here waits for the loads,
// so that a group's loads are in flight together whatever byte its rows start at (byte
// loads joined on the spot cost 3000 clocks a tile where a row has three scales).
__device__ __forceinline__ void load_e8m0_x4(const uint8_t *p, size_t i, int last, uint32_t &r0, uint32_t &r1,
                                             uint32_t &shifts) {
    const uintptr_t q = reinterpret_cast<uintptr_t>(p + i);
    const uint32_t *w = reinterpret_cast<const uint32_t *>(q & ~(uintptr_t)3);
    const uint32_t skip = (uint32_t)q & 3u;
    r0 = load_now(w);
    r1 = skip + (uint32_t)min(last, 3) > 3u ? load_now(w + 1) : 0u;
    shifts = shifts << 5 | skip << 3;
}
// field: 0 for the last one loaded, 1 for the one before, ...
__device__ __forceinline__ uint32_t e8m0_word(uint32_t r0, uint32_t r1, uint32_t shifts, int field) {
    return __funnelshift_r(r0, r1, shifts >> (5 * field));  // (by the low five bits)
}

#endif  // __CUDACC__

}  // namespace moe
