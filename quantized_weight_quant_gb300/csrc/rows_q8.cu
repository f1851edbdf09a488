// Rows to 8 bits: RMSNorm with an optional residual, or plain rows, written as
// E4M3 bytes with one f32 scale per row.
//     h = x + r,  v = h * w / sqrt(mean h^2 + eps)      (plain rows: v = x)
//     s = max(max |v| / 448, 2^-126),  code = e4m3(v / s)
// One pass over memory: a row's values stay in registers between the two
// reductions and the write.  max |h w| and sum h^2 are reduced together, since
// dividing by the row's one positive root keeps the order of the magnitudes
// (rounding is monotone), so the row's scale needs no second reduction.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qwq_internal.h"

namespace qwq {
namespace {

constexpr float kMax8 = 448.f;                    // largest E4M3 value
constexpr float kMinScale = 1.17549435e-38f;      // 2^-126

template <class T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two E4M3 bytes (lo in the low byte), nearest even, saturating, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight consecutive values; VEC: 16-byte aligned.
template <class T, bool VEC>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
    if constexpr (VEC && sizeof(T) == 4) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else if constexpr (VEC) {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        const T *e = reinterpret_cast<const T *>(&a);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = to_f<T>(e[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = to_f<T>(p[j]);
    }
}

template <class T, bool VEC>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
    if constexpr (VEC && sizeof(T) == 4) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if constexpr (VEC) {
        uint4 a;
        T *e = reinterpret_cast<T *>(&a);
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = from_f<T>(v[j]);
        *reinterpret_cast<uint4 *>(p) = a;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = from_f<T>(v[j]);
    }
}

// One block per row; a row longer than the registers hold is read again.
constexpr int kThreads = 256;

template <class T>
__global__ void __launch_bounds__(kThreads) rows_q8_kernel(const RowsQ8 a) {
    __shared__ float red_s[kThreads / 32];
    __shared__ unsigned red_m[kThreads / 32];
    const long long row = blockIdx.x;
    const int tid = threadIdx.x;
    const T *x = (const T *)a.x + row * a.ldx;
    const T *r = a.r ? (const T *)a.r + row * a.ldr : nullptr;
    T *h = a.h ? (T *)a.h + row * a.ldh : nullptr;
    uint8_t *y = a.y8 + row * a.ld8;
    float ss = 0.f;
    unsigned m = 0;
    for (int d = tid; d < a.D; d += kThreads) {
        const float v = r ? to_f<T>(x[d]) + to_f<T>(r[d]) : to_f<T>(x[d]);
        ss += v * v;
        m = max(m, __float_as_uint(a.w ? v * a.w[d] : v) & 0x7FFFFFFFu);   // magnitudes order as their bits, NaN last
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if ((tid & 31) == 0) red_s[tid >> 5] = ss, red_m[tid >> 5] = m;
    __syncthreads();
    ss = 0.f, m = 0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) ss += red_s[k], m = max(m, red_m[k]);
    const float root = a.w ? sqrtf(ss / (float)a.D + a.eps) : 1.f;
    const float top = __uint_as_float(m) / root / kMax8;
    const float s = top < kMinScale ? kMinScale : top;                     // a NaN stays
    if (tid == 0) a.ys[row] = s;
    for (int d = tid; d < a.D; d += kThreads) {
        const float v = r ? to_f<T>(x[d]) + to_f<T>(r[d]) : to_f<T>(x[d]);
        if (h) h[d] = from_f<T>(v);                                        // after this thread's last read of x[d], r[d]
        const float u = a.w ? v * a.w[d] / root : v;
        y[d] = (uint8_t)e4m3x2(u / s, 0.f);
    }
}

template <class T>
cudaError_t run(const RowsQ8 &a, cudaStream_t st) {
    rows_q8_kernel<T><<<a.S, kThreads, 0, st>>>(a);
    count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows_q8(const RowsQ8 &a, cudaStream_t st) {
    switch (a.type) {
    case B200Q_T_F32: return run<float>(a, st);
    case B200Q_T_F16: return run<__half>(a, st);
    default: return run<__nv_bfloat16>(a, st);
    }
}

}  // namespace qwq
