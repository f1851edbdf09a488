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

// A 16-byte vector of T as floats, and back.
template <class T> constexpr int kVec = 16 / (int)sizeof(T);

template <class T>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[kVec<T>]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const T *e = reinterpret_cast<const T *>(&a);
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) v[j] = to_f<T>(e[j]);
}

template <class T>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[kVec<T>]) {
    uint4 a;
    T *e = reinterpret_cast<T *>(&a);
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) e[j] = from_f<T>(v[j]);
    *reinterpret_cast<uint4 *>(p) = a;
}

// Sum and maximum over the block.
__device__ __forceinline__ void block_reduce(float &ss, unsigned &m) {
    __shared__ float red_s[32];
    __shared__ unsigned red_m[32];
    const int warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if (warps == 1) return;
    if ((threadIdx.x & 31) == 0) red_s[threadIdx.x >> 5] = ss, red_m[threadIdx.x >> 5] = m;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    ss = lane < warps ? red_s[lane] : 0.f;
    m = lane < warps ? red_m[lane] : 0u;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
}

// The row's root (1 for plain rows) and scale from the two reductions.
__device__ __forceinline__ void row_scale(const RowsQ8 &a, float ss, unsigned m, float &root, float &s) {
    root = a.w ? sqrtf(ss / (float)a.D + a.eps) : 1.f;
    const float top = __uint_as_float(m) / root / kMax8;
    s = top < kMinScale ? kMinScale : top;                     // a NaN stays
}

__device__ __forceinline__ unsigned magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }   // orders as |v|, NaN last

// One block per row, the row in registers: NV vectors of 16 bytes per thread
// (VEC: every operand's rows start on 16 bytes), or as many single values
// with the block's threads on neighbouring columns.
template <class T, int NV, bool VEC, bool NORM>
__global__ void __launch_bounds__(1024) rows_q8_kernel(const RowsQ8 a) {
    constexpr int E = kVec<T>;
    const long long row = blockIdx.x;
    const int tid = threadIdx.x, n = blockDim.x;
    const T *x = (const T *)a.x + row * a.ldx;
    const T *r = NORM && a.r ? (const T *)a.r + row * a.ldr : nullptr;
    T *h = NORM && a.h ? (T *)a.h + row * a.ldh : nullptr;
    uint8_t *y = a.y8 + row * a.ld8;
    float v[NV][E], g[NORM ? NV : 1][E];
    auto col = [&](int k, int j) { return VEC ? (k * n + tid) * E + j : (k * E + j) * n + tid; };
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if (VEC && col(k, E - 1) < a.D) {
            load_vec<T>(x + col(k, 0), v[k]);
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j) v[k][j] = col(k, j) < a.D ? to_f<T>(x[col(k, j)]) : 0.f;
        }
    }
    if (NORM && r) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float q[E];
            if (VEC && col(k, E - 1) < a.D) {
                load_vec<T>(r + col(k, 0), q);
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j) q[j] = col(k, j) < a.D ? to_f<T>(r[col(k, j)]) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < E; ++j) v[k][j] += q[j];
        }
    }
    float ss = 0.f;
    unsigned m = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if constexpr (NORM) {
            if (VEC && col(k, E - 1) < a.D) {
#pragma unroll
                for (int j = 0; j < E; j += 4) {
                    const float4 w = *reinterpret_cast<const float4 *>(a.w + col(k, j));
                    g[k][j] = w.x, g[k][j + 1] = w.y, g[k][j + 2] = w.z, g[k][j + 3] = w.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j) g[k][j] = col(k, j) < a.D ? a.w[col(k, j)] : 0.f;
            }
        }
        if (h) {
            if (VEC && col(k, E - 1) < a.D) {
                store_vec<T>(h + col(k, 0), v[k]);
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if (col(k, j) < a.D) h[col(k, j)] = from_f<T>(v[k][j]);
            }
        }
#pragma unroll
        for (int j = 0; j < E; ++j) {
            if constexpr (NORM) {
                ss = fmaf(v[k][j], v[k][j], ss);
                v[k][j] *= g[k][j];
            }
            m = max(m, magnitude(v[k][j]));
        }
    }
    block_reduce(ss, m);
    float root, s;
    row_scale(a, ss, m, root, s);
    if (tid == 0) a.ys[row] = s;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        uint32_t c[E];
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            const float u0 = NORM ? v[k][j] / root : v[k][j], u1 = NORM ? v[k][j + 1] / root : v[k][j + 1];
            const uint32_t p = e4m3x2(u0 / s, u1 / s);
            c[j] = p & 255u, c[j + 1] = p >> 8;
        }
        if (VEC && col(k, E - 1) < a.D) {
            const uint32_t lo = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
            if constexpr (E == 4) *reinterpret_cast<uint32_t *>(y + col(k, 0)) = lo;
            else *reinterpret_cast<uint2 *>(y + col(k, 0)) = make_uint2(lo, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (col(k, j) < a.D) y[col(k, j)] = (uint8_t)c[j];
        }
    }
}

// Rows longer than a block's registers hold: read twice.
constexpr int kLongThreads = 1024;

template <class T>
__global__ void __launch_bounds__(kLongThreads) rows_q8_long_kernel(const RowsQ8 a) {
    const long long row = blockIdx.x;
    const T *x = (const T *)a.x + row * a.ldx;
    const T *r = a.r ? (const T *)a.r + row * a.ldr : nullptr;
    T *h = a.h ? (T *)a.h + row * a.ldh : nullptr;
    uint8_t *y = a.y8 + row * a.ld8;
    float ss = 0.f;
    unsigned m = 0;
    for (int d = threadIdx.x; d < a.D; d += kLongThreads) {
        const float v = r ? to_f<T>(x[d]) + to_f<T>(r[d]) : to_f<T>(x[d]);
        ss = fmaf(v, v, ss);
        m = max(m, magnitude(a.w ? v * a.w[d] : v));
    }
    block_reduce(ss, m);
    float root, s;
    row_scale(a, ss, m, root, s);
    if (threadIdx.x == 0) a.ys[row] = s;
    for (int d = threadIdx.x; d < a.D; d += kLongThreads) {
        const float v = r ? to_f<T>(x[d]) + to_f<T>(r[d]) : to_f<T>(x[d]);
        if (h) h[d] = from_f<T>(v);                             // after this thread's last read of x[d], r[d]
        const float u = a.w ? v * a.w[d] / root : v;
        y[d] = (uint8_t)e4m3x2(u / s, 0.f);
    }
}

template <class T, int NV, bool VEC>
void start(const RowsQ8 &a, int threads, cudaStream_t st) {
    if (a.w) rows_q8_kernel<T, NV, VEC, true><<<a.S, threads, 0, st>>>(a);
    else rows_q8_kernel<T, NV, VEC, false><<<a.S, threads, 0, st>>>(a);
}

template <class T, bool VEC>
void start_nv(const RowsQ8 &a, int nv, int threads, cudaStream_t st) {
    switch (nv) {
    case 1: return start<T, 1, VEC>(a, threads, st);
    case 2: return start<T, 2, VEC>(a, threads, st);
    default: return start<T, 4, VEC>(a, threads, st);
    }
}

template <class T>
cudaError_t run(const RowsQ8 &a, cudaStream_t st) {
    constexpr int E = kVec<T>;
    auto ok = [](const void *p, long long ld) {
        return !p || ((uintptr_t)p % 16 == 0 && ld * (long long)sizeof(T) % 16 == 0);
    };
    const bool vec = ok(a.x, a.ldx) && ok(a.r, a.ldr) && ok(a.h, a.ldh) && (uintptr_t)a.w % 16 == 0;
    // few rows: one vector per thread, the shortest chain; many: several, so
    // that a block has more bytes in flight behind its one barrier
    const int units = (a.D + E - 1) / E;
    int dev = 0;
    cudaGetDevice(&dev);
    int nv = a.S <= 2 * sm_count(dev) ? 1 : 4;
    while (nv < 4 && units > nv * 1024) nv *= 2;
    if (units > nv * 1024) {
        rows_q8_long_kernel<T><<<a.S, kLongThreads, 0, st>>>(a);
    } else {
        const int threads = ((units + nv - 1) / nv + 31) / 32 * 32;
        if (vec) start_nv<T, true>(a, nv, threads, st);
        else start_nv<T, false>(a, nv, threads, st);
    }
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
