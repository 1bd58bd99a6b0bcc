// tcgen05 helpers of the bf16 attention beside those of gdn_tc.cuh: kind::f16
// products with bf16 operands, an MN-major operand, wide tensor-memory stores.
// Inline PTX only.
#pragma once

#include "gdn_tc.cuh"

namespace gdntc {

// Descriptor of an MN-major tile of 16-bit values (rows along K, 64 values of
// M or N in a row's 128 bytes) with the 128-byte swizzle: `block` bytes from
// one 64-value block of M or N to the next, 1024 bytes from 8 rows to the next
// 8. One MMA step consumes K = 16 rows, 2048 bytes of each block.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(unsigned saddr, unsigned block) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(block >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Instruction descriptor of kind::f16: f32 accumulator, bf16 A (K-major) and
// bf16 B (K-major, or MN-major), M x N.
__host__ __device__ constexpr unsigned idesc_bf16(unsigned M, unsigned N, bool b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// D (+)= A B, kind::f16 with bf16 operands, K = 16 a step. A lies in tensor
// memory, two values in a 32-bit column; B in shared memory.
__device__ __forceinline__ void mma_bf16_ts(unsigned d_tmem, unsigned a_tmem, uint64_t b_desc, unsigned idesc,
                                            bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// Warp-collective: 32 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tmem_st32(unsigned taddr, const unsigned (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

}  // namespace gdntc
