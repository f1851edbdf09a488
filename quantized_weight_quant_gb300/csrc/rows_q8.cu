// Rows to 8 bits: RMSNorm with an optional residual, or plain rows, written as
// E4M3 bytes with one f32 scale per row.
//     h = x + r,  v = h * w / sqrt(mean h^2 + eps)      (plain rows: v = x)
//     s = max(max |v| / 448, 2^-126),  code = e4m3(v / s)
// One pass over memory: a row's values stay in registers between the two
// reductions and the write.  max |h w| and sum h^2 are reduced together, since
// dividing by the row's one positive root keeps the order of the magnitudes
// (rounding is monotone), so the row's scale needs no second reduction.
// Bound: HBM for long batches (8192 x 12288 f32 80.5 us, 6250 GB/s); the rounds of
// blocks for a prompt (1571 x 6144 bf16 with residual 15.6 us, 4320 GB/s: five
// blocks of 192 threads fit on an SM, so the last 51 rows are a third round of
// their own); a call's latency for a few rows (3.5-4 us for 1 to 4 rows in a
// graph); the integer pipe where rows have to be shifted into place (6007 x 5003
// f16 36.5 us, plain rows 28.7 us).
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

// 16 bytes of T, and as floats.
template <class T> constexpr int kVec = 16 / (int)sizeof(T);
template <class T> union Vec {
    uint4 q;
    T e[kVec<T>];
    __device__ __forceinline__ float at(int j) const { return to_f<T>(e[j]); }
};

// v / d, correctly rounded, for a divisor that many values share: with
// rd = 1 / d rounded, q = v rd and one correction by the exact remainder
// (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  v / d itself, with its own reciprocal for
// every value, made these kernels arithmetic-bound.
__device__ __forceinline__ float div_by(float v, float d, float rd) {
    const float q = v * rd;
    return fmaf(fmaf(-q, d, v), rd, q);
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

// A plain row's scale from its largest magnitude.
__device__ __forceinline__ float plain_scale(unsigned m) {
    const float top = __uint_as_float(m) / kMax8;
    return top < kMinScale ? kMinScale : top;                  // a NaN stays
}

// A norm's scale from sum h^2 and max |h w|, and the factors f.x, f.y of h w
// that give the codes: (h w / root) / s = h w * 448 / max |h w|, one rounding
// instead of two divisions; where that factor could overflow, or the scale is
// the least one, 1 / root and 1 / s.  A sum that is not finite (a NaN or an
// infinity in the row, or h^2 beyond f32) makes the scale NaN.
__device__ __forceinline__ void norm_scale(const RowsQ8 &a, float ss, float m, float &s, float2 &f) {
    const float root = sqrtf(ss / (float)a.D + a.eps);
    const float top = ss <= 3.402823466e38f ? m / root / kMax8 : __int_as_float(0x7FC00000);
    s = top < kMinScale ? kMinScale : top;
    f = top < kMinScale || m < 1e-30f ? make_float2(1.f / root, 1.f / s) : make_float2(kMax8 / m, 1.f);
}

__device__ __forceinline__ unsigned magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }   // orders as |v|, NaN last

// The larger, or NaN if either is one (fmaxf drops a NaN: a weight that is one
// would leave the scale finite).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The 16 bytes from offset sh (0..15) on of two neighbouring vectors.  sh is
// the same for all vectors of a row.
__device__ __forceinline__ uint4 shifted(const uint4 &lo, const uint4 &hi, uint32_t sh) {
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const bool s8 = sh & 8, s4 = sh & 4;
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = s8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = s4 ? w[i + 1] : w[i];
    const uint32_t bits = 8 * (sh & 3);
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// A thread's values: vector k is kVec neighbouring columns from at(k) on, so
// that its bytes of y8 are aligned; a row's last vector may be short.
// ALIGNED: every wide operand's rows start on 16 bytes.  Otherwise a vector is
// the two aligned ones around it, shifted into place; next to the ends of a
// row, where those would reach past it, values are read one by one.  h is
// written in aligned vectors too (6007 x 5003 bf16 with residual: 71 us, value by
// value 98 us).
template <class T, bool ALIGNED> struct Cols {
    int n, tid, D;
    __device__ __forceinline__ int at(int k) const { return (k * n + tid) * kVec<T>; }
    __device__ __forceinline__ bool full(int k) const { return at(k) + kVec<T> <= D; }
    template <class U, bool AL = ALIGNED>
    __device__ __forceinline__ Vec<U> load(const U *p, int c) const {
        constexpr int m = kVec<U>;
        Vec<U> v;
        if (AL ? c + m <= D : c >= m && c + 2 * m <= D) {
            const char *a = (const char *)(p + c);
            const uint32_t sh = AL ? 0u : (uint32_t)((uintptr_t)a & 15u);
            const uint4 *b = reinterpret_cast<const uint4 *>(a - sh);
            v.q = AL ? b[0] : shifted(b[0], b[1], sh);
        } else {
#pragma unroll
            for (int j = 0; j < m; ++j) v.e[j] = c + j < D ? p[c + j] : from_f<U>(0.f);
        }
        return v;
    }
    // Called by whole warps.  Unaligned rows: a lane writes the aligned 16 bytes
    // that begin in its left neighbour's vector; the warp's first and last lanes,
    // and the row's last, write what is left of theirs value by value.
    __device__ __forceinline__ void store(T *p, int k, const Vec<T> &v) const {
        constexpr int m = kVec<T>;
        const int c = at(k);
        const bool f = full(k);
        const uint32_t sh = ALIGNED ? 0u : (uint32_t)((uintptr_t)(p + c) & 15u);
        int lo = 0, hi = m;                       // values outside lo .. hi-1 are written one by one
        if (sh == 0) {
            if (f) *reinterpret_cast<uint4 *>(p + c) = v.q;
        } else {
            const uint4 left = make_uint4(__shfl_up_sync(0xffffffffu, v.q.x, 1), __shfl_up_sync(0xffffffffu, v.q.y, 1),
                                          __shfl_up_sync(0xffffffffu, v.q.z, 1), __shfl_up_sync(0xffffffffu, v.q.w, 1));
            const int lane = threadIdx.x & 31, split = m - (int)(sh / sizeof(T));
            if (lane == 0) lo = split;
            if (lane == 31 || c + 2 * m > D) hi = split;
            if (f && lane != 0) *reinterpret_cast<uint4 *>((char *)(p + c) - sh) = shifted(left, v.q, 16 - sh);
        }
        if (ALIGNED && f) return;
#pragma unroll
        for (int j = 0; j < m; ++j)
            if (c + j < D && (!f || j < lo || j >= hi)) p[c + j] = v.e[j];
    }
    // E4M3 bytes, in pairs
    __device__ __forceinline__ void store8(uint8_t *y, int k, const uint32_t (&c)[kVec<T> / 2]) const {
        if (full(k)) {
            const uint32_t lo = __byte_perm(c[0], c[1], 0x5410);
            if constexpr (kVec<T> == 4) *reinterpret_cast<uint32_t *>(y + at(k)) = lo;
            else *reinterpret_cast<uint2 *>(y + at(k)) = make_uint2(lo, __byte_perm(c[2], c[3], 0x5410));
        } else {
#pragma unroll
            for (int j = 0; j < kVec<T>; ++j)
                if (at(k) + j < D) y[at(k) + j] = (uint8_t)(c[j / 2] >> (8 * (j & 1)));
        }
    }
};

// Threads of a block at most, by vectors per thread: registers for two blocks
// per SM at least, so that one row's loads run under another's arithmetic.
constexpr int most_threads(int nv) { return nv == 1 ? 1024 : 512; }
constexpr int least_blocks(int nv) { return nv == 1 ? 1 : 2; }

// The row in registers, NV vectors per thread; blockDim.y rows per block (more
// than one only where blockDim.x is one warp).
template <class T, int NV, bool ALIGNED>
__global__ void __launch_bounds__(most_threads(NV), least_blocks(NV)) quantize_q8_kernel(const RowsQ8 a) {
    constexpr int E = kVec<T>;
    const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= a.S) return;                      // whole warps: blockDim.y > 1 has no barrier
    const Cols<T, ALIGNED> cols{(int)blockDim.x, (int)threadIdx.x, a.D};
    const T *x = (const T *)a.x + row * a.ldx;
    uint8_t *y = a.y8 + row * a.ld8;
    Vec<T> v[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] = cols.load(x, cols.at(k));
    unsigned m = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < E; ++j) m = max(m, magnitude(v[k].at(j)));
    float none = 0.f;
    block_reduce(none, m);
    const float s = plain_scale(m), rs = 1.f / s;
    if (threadIdx.x == 0) a.ys[row] = s;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        uint32_t c[E / 2];
#pragma unroll
        for (int j = 0; j < E; j += 2) c[j / 2] = e4m3x2(div_by(v[k].at(j), s, rs), div_by(v[k].at(j + 1), s, rs));
        cols.store8(y, k, c);
    }
}

// RES: with r or h.  Without either it keeps no sum's operands and no rounded
// copy (8192 x 12288 f32: 91 us, with the code for both in place 151 us; 6007 x
// 5003 f16 36.5 and 44.4 us).
template <class T, int NV, bool ALIGNED, bool RES>
__global__ void __launch_bounds__(most_threads(NV), least_blocks(NV)) rmsnorm_q8_kernel(const RowsQ8 a) {
    constexpr int E = kVec<T>;
    const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= a.S) return;
    const Cols<T, ALIGNED> cols{(int)blockDim.x, (int)threadIdx.x, a.D};
    const T *x = (const T *)a.x + row * a.ldx;
    const T *r = RES && a.r ? (const T *)a.r + row * a.ldr : nullptr;
    T *h = RES && a.h ? (T *)a.h + row * a.ldh : nullptr;
    uint8_t *y = a.y8 + row * a.ld8;
    Vec<T> xv[NV], rv[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) xv[k] = cols.load(x, cols.at(k));
    if (r) {
#pragma unroll
        for (int k = 0; k < NV; ++k) rv[k] = cols.load(r, cols.at(k));
    }
    const bool w16 = ALIGNED || (uintptr_t)a.w % 16 == 0;      // its one row needs no shift where x's rows do
    float v[NV][E], ss = 0.f, m = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        Vec<T> hv;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            v[k][j] = r ? xv[k].at(j) + rv[k].at(j) : xv[k].at(j);
            hv.e[j] = from_f<T>(v[k][j]);
        }
        if (h) cols.store(h, k, hv);
        float g[E];
#pragma unroll
        for (int j = 0; j < E; j += 4) {
            const Vec<float> wv = w16 ? cols.template load<float, true>(a.w, cols.at(k) + j)
                                      : cols.template load<float, false>(a.w, cols.at(k) + j);
#pragma unroll
            for (int i = 0; i < 4; ++i) g[j + i] = wv.e[i];
        }
#pragma unroll
        for (int j = 0; j < E; ++j) {
            ss = fmaf(v[k][j], v[k][j], ss);
            v[k][j] *= g[j];
            m = max_nan(m, fabsf(v[k][j]));
        }
    }
    unsigned mb = __float_as_uint(m);
    block_reduce(ss, mb);
    float s;
    float2 f;
    norm_scale(a, ss, __uint_as_float(mb), s, f);
    if (threadIdx.x == 0) a.ys[row] = s;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        uint32_t c[E / 2];
#pragma unroll
        for (int j = 0; j < E; j += 2) c[j / 2] = e4m3x2(v[k][j] * f.x * f.y, v[k][j + 1] * f.x * f.y);
        cols.store8(y, k, c);
    }
}

// Rows longer than a block's registers hold (16384 values of 16 bits or f32):
// read twice, value by value (1571 x 28672 bf16: plain rows 52.6 us, 2570 GB/s of
// one pass; the norm with residual 183 us).
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
    const unsigned D = a.D;                      // d passes 2^31 - 1 by up to a block
    for (unsigned d = threadIdx.x; d < D; d += kLongThreads) {
        const float v = r ? to_f<T>(x[d]) + to_f<T>(r[d]) : to_f<T>(x[d]);
        ss = fmaf(v, v, ss);
        m = max(m, magnitude(a.w ? v * a.w[d] : v));
    }
    block_reduce(ss, m);
    float s = plain_scale(m);
    float2 f = make_float2(0.f, 0.f);
    if (a.w) norm_scale(a, ss, __uint_as_float(m), s, f);
    if (threadIdx.x == 0) a.ys[row] = s;
    const float rs = 1.f / s;
    for (unsigned d = threadIdx.x; d < D; d += kLongThreads) {
        const float v = r ? to_f<T>(x[d]) + to_f<T>(r[d]) : to_f<T>(x[d]);
        if (h) h[d] = from_f<T>(v);                             // after this thread's last read of x[d], r[d]
        y[d] = (uint8_t)e4m3x2(a.w ? v * a.w[d] * f.x * f.y : div_by(v, s, rs), 0.f);
    }
}

template <class T, int NV, bool ALIGNED>
void start(const RowsQ8 &a, dim3 block, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.S + (long long)block.y - 1) / block.y);
    if (a.w && (a.r || a.h)) rmsnorm_q8_kernel<T, NV, ALIGNED, true><<<grid, block, 0, st>>>(a);
    else if (a.w) rmsnorm_q8_kernel<T, NV, ALIGNED, false><<<grid, block, 0, st>>>(a);
    else quantize_q8_kernel<T, NV, ALIGNED><<<grid, block, 0, st>>>(a);
}

template <class T, bool ALIGNED>
void start_nv(const RowsQ8 &a, int nv, dim3 block, cudaStream_t st) {
    if (nv == 1) start<T, 1, ALIGNED>(a, block, st);
    else if (nv == 2) start<T, 2, ALIGNED>(a, block, st);
    else if (nv == 4 || kVec<T> == 8) start<T, 4, ALIGNED>(a, block, st);
    else start<T, 32 / kVec<T>, ALIGNED>(a, block, st);
}

template <class T>
cudaError_t run(const RowsQ8 &a, cudaStream_t st) {
    constexpr int E = kVec<T>;
    auto ok = [](const void *p, long long ld) {
        return !p || ((uintptr_t)p % 16 == 0 && ld * (long long)sizeof(T) % 16 == 0);
    };
    const bool aligned = ok(a.x, a.ldx) && ok(a.r, a.ldr) && ok(a.h, a.ldh) && (uintptr_t)a.w % 16 == 0;
    const int units = (int)((a.D + (E - 1ll)) / E);           // 16-byte vectors of a row
    int dev = 0;
    cudaGetDevice(&dev);
    // Few rows: as many threads as there are vectors, the shortest chain (6144
    // bf16 with residual: 1 row 3.7-4.0 us, 128 rows 4.5 us; with 256 threads at
    // most 4.75 and 5.35 us; 4 rows of 12288, no residual, 3.5 and 3.3 us).
    // Many: up to 32 values per thread in blocks of 256, several per SM (1571
    // rows of 6144 bf16 with residual 15.8 us; with 1024 threads 19.3 us).
    int nv = 1;
    const int most = a.S <= 2 * sm_count(dev) ? 1024 : 256;
    while (nv < 32 / E && units > nv * (most < most_threads(nv) ? most : most_threads(nv))) nv *= 2;
    dim3 block(((units + nv - 1) / nv + 31) / 32 * 32);
    // many short rows: a warp each, four to a block, no barrier (16000 rows of 64
    // f32 4.9 us, of 512 bf16 with residual 12.2 us; a block each 10.4 and 13.7 us)
    if (a.S > 2 * sm_count(dev) && units <= 128) {
        nv = units <= 32 ? 1 : units <= 64 ? 2 : 4;
        block = dim3(32, 4);
    }
    if ((int)block.x > most_threads(nv)) {
        rows_q8_long_kernel<T><<<a.S, kLongThreads, 0, st>>>(a);
    } else if (aligned) {
        start_nv<T, true>(a, nv, block, st);
    } else {
        start_nv<T, false>(a, nv, block, st);
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
