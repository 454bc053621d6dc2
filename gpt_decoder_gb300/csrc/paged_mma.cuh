// Pieces of the kernels that take the paged cache's rows straight into matrix-instruction registers: the
// instruction, the exponential, and 8-bit codes as bf16.
#pragma once

#include "launch.cuh"

namespace gk {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// D += A B, bf16 operands, float32 accumulators: A 16x16, B 16x8.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The codes in bytes 0 and 2 of x as a pair of bf16.
__device__ __forceinline__ uint32_t codes02(const CodeMasks& k, uint32_t x) {
    const uint32_t a = and_or(x, k.low7, k.bf16_128), b = and_or(x, k.sign, k.bf16_128);
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&d);
}
// Codes 0 and 1 (or 2 and 3) of a word as a pair of bf16: 128 + the low seven bits, less 128 or 256.
__device__ __forceinline__ uint32_t codes_pair(const CodeMasks& k, uint32_t w, int second) {
    return codes02(k, __byte_perm(w, 0, second ? 0x4342 : 0x4140));
}

}  // namespace gk
