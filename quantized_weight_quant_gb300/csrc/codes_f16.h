// Weight codes as exact f16 operands of the warp-level tensor instruction
// m16n8k16, for the kernels that stream weights (qmv_q8.cu, moe_experts.cu).
#pragma once

#include <cuda_fp16.h>

#include "qwq_internal.h"

namespace qwq {

// KC: codes in 16 bytes.  MMAS: instructions per 32-bit word of codes (each
// takes four codes per thread and row).
template <int FMT> struct Fmt;
template <> struct Fmt<B200Q_I8> { static constexpr int KC = 16, MMAS = 1; };
template <> struct Fmt<B200Q_I4> { static constexpr int KC = 32, MMAS = 2; };
template <> struct Fmt<B200Q_I2> { static constexpr int KC = 64, MMAS = 4; };

__device__ __forceinline__ uint32_t lop_or(uint32_t w, uint32_t mask) {     // (w & mask) | 1024 in f16, twice
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(0x64006400u));
    return r;
}

__device__ __forceinline__ uint32_t fma_h2(uint32_t a, uint32_t mul, uint32_t add) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(mul), "r"(add));
    return r;
}

// Instruction t of a word of codes: two pairs of exact f16 values.
//   int8  (0,1) (2,3);  int4  t = 0: (0,4) (2,6), t = 1: (1,5) (3,7);
//   int2  (t,8+t) (4+t,12+t)
// A field at bit b of 1024's mantissa is 1024 + c 2^b; times 2^-b, minus the
// rest and the zero point, is the code's value.
template <int FMT>
__device__ __forceinline__ void fields(uint32_t w, int t, uint32_t &a, uint32_t &b) {
    constexpr uint32_t one = 0x3C003C00u;
    if constexpr (FMT == B200Q_I8) {                      // 1024 + (c + 128) - 1152
        const uint32_t u = w ^ 0x80808080u;
        a = fma_h2(__byte_perm(u, 0x64006400u, 0x5150), one, 0xE480E480u);
        b = fma_h2(__byte_perm(u, 0x64006400u, 0x5352), one, 0xE480E480u);
    } else if constexpr (FMT == B200Q_I4) {               // - 1032, / 16 - 72
        const uint32_t mask = t ? 0x00F000F0u : 0x000F000Fu;
        const uint32_t mul = t ? 0x2C002C00u : one, add = t ? 0xD480D480u : 0xE408E408u;
        a = fma_h2(lop_or(w, mask), mul, add);
        b = fma_h2(lop_or(w >> 8, mask), mul, add);
    } else {                                              // - 1026, / 4 - 258, / 16 - 66, / 64 - 18
        const uint32_t mask = 0x00030003u << (2 * t);
        const uint32_t mul = t == 0 ? one : t == 1 ? 0x34003400u : t == 2 ? 0x2C002C00u : 0x24002400u;
        const uint32_t add = t == 0 ? 0xE402E402u : t == 1 ? 0xDC08DC08u : t == 2 ? 0xD420D420u : 0xCC80CC80u;
        a = fma_h2(lop_or(w, mask), mul, add);
        b = fma_h2(lop_or(w >> 8, mask), mul, add);
    }
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

}  // namespace qwq
