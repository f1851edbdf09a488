// The experts' layer for a few tokens, routed on the device.
//     h[s,j] = act(gate_e x[s]) * (up_e x[s]),   y[s] = res[s] + sum_j wts[s,j] down_e h[s,j],   e = ids[s,j]
// One warp per (slot, row of gate and up), then one per (token, row of down),
// lanes over the bytes of a row of codes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qmat_q8.h"
#include "qwq_internal.h"

namespace qwq {
namespace {

constexpr int kWarps = 8;

__device__ unsigned int g_moe_err = 0;        // first error a kernel recorded (a B200Q_E* code, negated)

// Code j of a byte, as its value.
template <int FMT> __device__ __forceinline__ float value(uint8_t b, int j) {
    if constexpr (FMT == B200Q_I8) return (float)(int8_t)b;
    if constexpr (FMT == B200Q_I4) return (float)((b >> (4 * j)) & 15) - 8.f;
    return (float)((b >> (2 * j)) & 3) - 2.f;
}
template <int FMT> constexpr int kPerByte = FMT == B200Q_I8 ? 1 : FMT == B200Q_I4 ? 2 : 4;

// The expert of a slot, or -1.
__device__ __forceinline__ int expert_at(const int *ids, long long at, int E) {
    const int e = ids[at];
    if (e >= 0 && e < E) return e;
    if (e != -1) atomicCAS(&g_moe_err, 0u, (unsigned)(-B200Q_EINVAL));
    return -1;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int FMT>
__global__ void __launch_bounds__(32 * kWarps) moe_up_kernel(const Moe p, const Experts ex, float *h) {
    const int f = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const long long at = blockIdx.y;
    const int e = expert_at(p.ids, at, ex.E);
    if (f >= ex.F || e < 0) return;
    const Expert &t = ex.table[e];
    const uint8_t *g = t.codes[0] + f * ex.ld_in, *u = t.codes[1] + f * ex.ld_in;
    float a = 0.f, b = 0.f;
    for (int i = lane * kPerByte<FMT>; i < ex.D; i += 32 * kPerByte<FMT>)
        for (int j = 0; j < kPerByte<FMT> && i + j < ex.D; ++j) {
            const float x = load_typed(p.x, at / p.k * p.ldx + i + j, p.type);
            a = fmaf(value<FMT>(g[i / kPerByte<FMT>], j), x, a);
            b = fmaf(value<FMT>(u[i / kPerByte<FMT>], j), x, b);
        }
    a = warp_sum(a) * t.scales[0][f], b = warp_sum(b) * t.scales[1][f];
    if (lane == 0) h[at * ex.F + f] = act_q8(a, p.act) * b;
}

template <int FMT>
__global__ void __launch_bounds__(32 * kWarps) moe_down_kernel(const Moe p, const Experts ex, const float *h) {
    const int o = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const long long s = blockIdx.y;
    if (o >= ex.D) return;
    float y = 0.f;
    for (int k = 0; k < p.k; ++k) {
        const int e = expert_at(p.ids, s * p.k + k, ex.E);
        if (e < 0) continue;
        const Expert &t = ex.table[e];
        const uint8_t *d = t.codes[2] + o * ex.ld_out;
        const float *hr = h + (s * p.k + k) * ex.F;
        float a = 0.f;
        for (int i = lane * kPerByte<FMT>; i < ex.F; i += 32 * kPerByte<FMT>)
            for (int j = 0; j < kPerByte<FMT> && i + j < ex.F; ++j)
                a = fmaf(value<FMT>(d[i / kPerByte<FMT>], j), hr[i + j], a);
        y = fmaf(p.wts[s * p.k + k], warp_sum(a) * t.scales[2][o], y);
    }
    if (lane == 0) {
        if (p.res) y += load_typed(p.res, s * p.ldr + o, p.type);
        store_typed(p.y, s * p.ldy + o, p.type, y);
    }
}

template <int FMT>
cudaError_t run(const Moe &a, cudaStream_t st) {
    const Experts &ex = *a.ex;
    const int part = 65535 / a.k;              // tokens per launch: slots are grid rows
    const int b = a.type == B200Q_T_F32 ? 4 : 2;
    float *h = nullptr;
    cudaError_t e = workspace_alloc((void **)&h, (size_t)(a.S < part ? a.S : part) * a.k * ex.F * 4, st);
    if (e != cudaSuccess) return e;
    for (int s0 = 0; s0 < a.S && e == cudaSuccess; s0 += part) {
        Moe c = a;
        c.S = a.S - s0 < part ? a.S - s0 : part;
        c.x = (const char *)a.x + s0 * a.ldx * b;
        c.ids = a.ids + (long long)s0 * a.k;
        c.wts = a.wts + (long long)s0 * a.k;
        c.res = a.res ? (const char *)a.res + s0 * a.ldr * b : nullptr;
        c.y = (char *)a.y + s0 * a.ldy * b;
        moe_up_kernel<FMT><<<dim3((ex.F + kWarps - 1) / kWarps, c.S * a.k), 32 * kWarps, 0, st>>>(c, ex, h);
        moe_down_kernel<FMT><<<dim3((ex.D + kWarps - 1) / kWarps, c.S), 32 * kWarps, 0, st>>>(c, ex, h);
        count_launch(2);
        e = cudaGetLastError();
    }
    cudaError_t e2 = workspace_free(h, st);
    return e != cudaSuccess ? e : e2;
}

}  // namespace

cudaError_t launch_moe_experts(const Moe &a, cudaStream_t st) {
    switch (a.ex->fmt) {
    case B200Q_I8: return run<B200Q_I8>(a, st);
    case B200Q_I4: return run<B200Q_I4>(a, st);
    default: return run<B200Q_I2>(a, st);
    }
}

// Reads and clears the error word (0: none).
cudaError_t moe_take_error(unsigned int *code) {
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_moe_err, sizeof(unsigned int));
    if (e == cudaSuccess && *code) e = cudaMemcpyToSymbol(g_moe_err, &zero, sizeof(unsigned int));
    return e;
}

}  // namespace qwq
