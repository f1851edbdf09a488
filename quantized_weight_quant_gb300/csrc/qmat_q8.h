// Shared by the 8-bit matmul kernels: the epilogue and its element types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qwq_internal.h"

namespace qwq {

// How a call is launched, from its sizes and the number of SMs alone (host
// arithmetic: what the launchers use and b200q_selftest_q8_plan reports).
struct MvPlan {                // the few-row kernel
    bool fits;                 // false: x does not fit in shared memory, or too many rows
    bool xh;                   // x staged in f16
    int ahead, warps, pitch, grid, tiles, ng;
    long long smem;
};
struct GemmPlan {              // one launch of the tcgen05 kernel
    bool ok;                   // false: more items than 32 bits number
    int N, n_tiles, nk;        // rows of x8 per tile, tiles along them, k-blocks
    int items, grid, grain, stages;
    long long tiles;
    bool cut;                  // some tile is shared by several CTAs
    long long plane_bytes;
    size_t smem;
};
MvPlan plan_mv_q8(int fmt, bool pair, int O, long long ld, int S, int n_sms);
GemmPlan plan_gemm_q8(int fmt, bool pair, int O, int I, int S, int n_sms);
int gemm_q8_part(int O, int I);         // rows of x8 per launch
int gemm_q8_parts(int S, int part);     // launches

// v, activated.  f32 expf / erff; for large |v| the exponentials
// overflow or vanish to the activation's limits.  __fdividef (2 ulp) gives 0
// where silu's denominator passes 2^126, v < -87, where silu is below 1e-36.
// Against 64 bits silu is 2.2e-7 off at most for v > -80 (with / instead 2.1e-7),
// gelu_tanh 1.3e-6 for v > -4.  Not /, whose slow path the epilogue would carry:
// the pair 12288 x 6144 over 1571 rows 215 us instead of 207, a gelu_tanh product
// of that size 157 instead of 120.
template <int ACT>
__device__ __forceinline__ float act_q8(float v) {
    if constexpr (ACT == B200Q_ACT_RELU) return v < 0.f ? 0.f : v;      // keeps a NaN
    if constexpr (ACT == B200Q_ACT_GELU) return 0.5f * v * (1.f + erff(v * 0.70710678f));
    if constexpr (ACT == B200Q_ACT_GELU_TANH)
        return __fdividef(v, 1.f + expf(-1.59576912f * (v + 0.044715f * v * v * v)));    // (1 + tanh a) / 2 = 1 / (1 + e^-2a)
    if constexpr (ACT == B200Q_ACT_SILU) return __fdividef(v, 1.f + expf(-v));
    return v;
}

// The first K of v.
template <int ACT, int K, int N>
__device__ __forceinline__ void act_n(float (&v)[N]) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = act_q8<ACT>(v[k]);
}

__device__ __forceinline__ float act_q8(float v, int act) {
    switch (act) {
    case B200Q_ACT_RELU: return act_q8<B200Q_ACT_RELU>(v);
    case B200Q_ACT_GELU: return act_q8<B200Q_ACT_GELU>(v);
    case B200Q_ACT_GELU_TANH: return act_q8<B200Q_ACT_GELU_TANH>(v);
    case B200Q_ACT_SILU: return act_q8<B200Q_ACT_SILU>(v);
    }
    return v;
}

__device__ __forceinline__ float load_typed(const void *p, long long i, int type) {
    if (type == B200Q_T_F32) return ((const float *)p)[i];
    if (type == B200Q_T_F16) return __half2float(((const __half *)p)[i]);
    return __bfloat162float(((const __nv_bfloat16 *)p)[i]);
}

__device__ __forceinline__ void store_typed(void *p, long long i, int type, float v) {
    if (type == B200Q_T_F32) ((float *)p)[i] = v;
    else if (type == B200Q_T_F16) ((__half *)p)[i] = __float2half_rn(v);
    else ((__nv_bfloat16 *)p)[i] = __float2bfloat16_rn(v);
}

}  // namespace qwq
