// From one block to the next: norm after, gate, scaled residual, norm before.
//     p = m [* w_post / rms(m)],  h' = res_scale h + out_scale gate p,  y = h' w / rms(h')
// A block per row, each pass over the row from memory again.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qwq_internal.h"

namespace qwq {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__half *p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float block_sum(float v) {
    __shared__ float red[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += red[w];
    return s;
}

template <class T, class Y>
__global__ void __launch_bounds__(kThreads) block_norm_kernel(const BlockNorm a) {
    const long long row = blockIdx.x;
    const T *m = (const T *)a.m + row * a.ldm;
    const T *h = a.h ? (const T *)a.h + row * a.ldh : nullptr;
    const T *g = a.gate ? (const T *)a.gate + row * a.ldg : nullptr;
    T *o = a.h_out ? (T *)a.h_out + row * a.ldo : nullptr;
    Y *y = a.y ? (Y *)a.y + row * a.ldy : nullptr;
    const unsigned D = a.D;
    float post = 1.f;
    if (a.w_post) {
        float ss = 0.f;
        for (unsigned d = threadIdx.x; d < D; d += kThreads) ss = fmaf(to_f(m[d]), to_f(m[d]), ss);
        post = 1.f / sqrtf(block_sum(ss) / (float)a.D + a.eps);
    }
    auto next = [&](unsigned d) {
        float p = to_f(m[d]);
        if (a.w_post) p = p * post * a.w_post[d];
        if (g) p *= to_f(g[a.gate_cols == 1 ? 0 : d]);
        return fmaf(a.out_scale, p, h ? a.res_scale * to_f(h[d]) : 0.f);
    };
    float rms = 0.f;
    if (y) {
        float ss = 0.f;
        for (unsigned d = threadIdx.x; d < D; d += kThreads) {
            const float v = next(d);
            ss = fmaf(v, v, ss);
        }
        rms = 1.f / sqrtf(block_sum(ss) / (float)a.D + a.eps);
    }
    for (unsigned d = threadIdx.x; d < D; d += kThreads) {
        const float v = next(d);               // before this thread's write of h_out[d], which may be h or m
        if (o) put(o + d, v);
        if (y) put(y + d, v * rms * a.w[d]);
    }
}

template <class T, class Y>
cudaError_t start(const BlockNorm &a, cudaStream_t st) {
    block_norm_kernel<T, Y><<<a.S, kThreads, 0, st>>>(a);
    count_launch();
    return cudaGetLastError();
}

template <class T>
cudaError_t run(const BlockNorm &a, cudaStream_t st) {
    switch (a.ytype) {
    case B200Q_T_F32: return start<T, float>(a, st);
    case B200Q_T_F16: return start<T, __half>(a, st);
    default: return start<T, __nv_bfloat16>(a, st);
    }
}

}  // namespace

cudaError_t launch_block_norm(const BlockNorm &a, cudaStream_t st) {
    switch (a.type) {
    case B200Q_T_F32: return run<float>(a, st);
    case B200Q_T_F16: return run<__half>(a, st);
    default: return run<__nv_bfloat16>(a, st);
    }
}

}  // namespace qwq
