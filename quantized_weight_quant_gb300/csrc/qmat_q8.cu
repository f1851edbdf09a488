// Matrix product and gated pair on 8-bit rows (E4M3 bytes, one f32 scale per
// row) with quantized weights and an epilogue:
//     y[s,o] = act(scale[o] xs[s] sum_i deq(W[o,i]) x8[s,i] + bias[o]) + res[s,o]
//     y[s,f] = act(g) u
#include <cuda_fp8.h>

#include "qmat_q8.h"

namespace qwq {
namespace {

constexpr int kTok = 4;      // tokens per warp

template <int FMT>
__device__ __forceinline__ float weight_at(const uint8_t *row, int i) {
    if (FMT == B200Q_I8) return (float)(int8_t)row[i];
    if (FMT == B200Q_I4) return (float)((row[i >> 1] >> (4 * (i & 1))) & 15) - 8.f;
    return (float)((row[i >> 2] >> (2 * (i & 3))) & 3) - 2.f;
}

__device__ __forceinline__ float e4m3_f(uint8_t c) {
    __nv_fp8_e4m3 v;
    v.__x = c;
    return (float)v;
}

// One warp per output column and four tokens.
template <int FMT, bool GLU>
__global__ void __launch_bounds__(256) mat_q8_kernel(const MatQ8 a, const uint8_t *cg, const float *sg,
                                                     const uint8_t *cu, const float *su, int O, int I, long long ld) {
    const int lane = threadIdx.x & 31;
    const int o = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int s0 = blockIdx.y * kTok;
    if (o >= O) return;
    float g[kTok] = {}, u[kTok] = {};
    for (int i = lane; i < I; i += 32) {
        const float wg = weight_at<FMT>(cg + o * ld, i), wu = GLU ? weight_at<FMT>(cu + o * ld, i) : 0.f;
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            if (s0 + t >= a.S) break;
            const float x = e4m3_f(a.x8[(s0 + t) * a.ld8 + i]);
            g[t] = fmaf(wg, x, g[t]);
            if (GLU) u[t] = fmaf(wu, x, u[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < kTok; ++t)
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) {
            g[t] += __shfl_xor_sync(0xffffffffu, g[t], k);
            u[t] += __shfl_xor_sync(0xffffffffu, u[t], k);
        }
    if (lane) return;
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
        const long long s = s0 + t;
        if (s >= a.S) break;
        const float xs = a.xs[s];
        float v = act_q8(g[t] * xs * sg[o] + (a.bias_g ? a.bias_g[o] : 0.f), a.act);
        if (GLU) v *= u[t] * xs * su[o] + (a.bias_u ? a.bias_u[o] : 0.f);
        if (a.res) v += load_typed(a.res, s * a.ldr + o, a.type);
        store_typed(a.y, s * a.ldy + o, a.type, v);
    }
}

template <int FMT>
cudaError_t run(const MatQ8 &a, cudaStream_t st) {
    const Tensor &t = *a.tg;
    const int blocks = (a.S + kTok - 1) / kTok;
    MatQ8 p = a;
    for (int b0 = 0; b0 < blocks; b0 += 65535) {
        dim3 grid((t.O + 7) / 8, blocks - b0 < 65535 ? blocks - b0 : 65535);
        if (a.tu)
            mat_q8_kernel<FMT, true><<<grid, 256, 0, st>>>(p, t.codes, t.scales, a.tu->codes, a.tu->scales, t.O, t.I, t.ld);
        else
            mat_q8_kernel<FMT, false><<<grid, 256, 0, st>>>(p, t.codes, t.scales, nullptr, nullptr, t.O, t.I, t.ld);
        count_launch();
        const long long n = 65535ll * kTok, b = a.type == B200Q_T_F32 ? 4 : 2;
        p.S -= (int)n;
        p.x8 += n * a.ld8;
        p.xs += n;
        p.y = (char *)p.y + n * a.ldy * b;
        if (p.res) p.res = (const char *)p.res + n * a.ldr * b;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mat_q8(const MatQ8 &a, cudaStream_t st) {
    if (a.S > 8) return launch_gemm_q8(a, st);
    switch (a.tg->fmt) {
    case B200Q_I8: return run<B200Q_I8>(a, st);
    case B200Q_I4: return run<B200Q_I4>(a, st);
    case B200Q_I2: return run<B200Q_I2>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace qwq
