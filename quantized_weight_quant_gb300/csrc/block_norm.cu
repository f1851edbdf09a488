// From one block to the next: norm after, gate, scaled residual, norm before.
//     p = m [* w_post / rms(m)],  h' = res_scale h + out_scale gate p,  y = h' w / rms(h')
// One pass over memory: a row's values stay in registers from the reads to the
// writes, through both sums.  Bound: HBM for many rows, a call's latency for few.
//   * Many rows: blocks walk them, and ask for the next row as soon as this one's
//     values are in f32, so that its reads run under the second sum and the writes.
//   * Rows that do not start on 16 bytes, but all operands' alike (one stride, odd):
//     the vectors are those of the memory, and the columns of a row begin inside the
//     first.  The weights, which then meet them at another place in every row, are
//     kept in shared memory (with a gate that is one row for all), the values of a
//     vector in rows of their own (no bank conflicts).  Operands that do not start alike are read value by value.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "launch.h"
#include "qwq_internal.h"

namespace qwq {
namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// VE neighbouring values, moved in pieces of at most 16 bytes.
template <int BYTES> struct Piece { using T = uint4; };
template <> struct Piece<8> { using T = uint2; };
template <> struct Piece<4> { using T = uint32_t; };
template <> struct Piece<2> { using T = unsigned short; };
template <class T, int VE> union Pack {
    using P = typename Piece<VE * (int)sizeof(T)>::T;
    static constexpr int kPieces = VE * (int)sizeof(T) / (int)sizeof(P);
    P q[kPieces];
    T e[VE];
    __device__ __forceinline__ Pack() {}
    __device__ __forceinline__ void get(const T *p) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) q[i] = reinterpret_cast<const P *>(p)[i];
    }
    // As get(), here and now: volatile, so that the compiler does not move the loads
    // of the next row to where they are used.
    __device__ __forceinline__ void fetch(const T *p) {
        if constexpr (sizeof(P) == 16) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(q[i].x), "=r"(q[i].y), "=r"(q[i].z), "=r"(q[i].w)
                             : "l"(p + i * (16 / (int)sizeof(T))));
        } else {
            get(p);
        }
    }
    __device__ __forceinline__ void put(T *p) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) reinterpret_cast<P *>(p)[i] = q[i];
    }
};

template <class T, int VE>
__device__ __forceinline__ void store(T *p, const float (&v)[VE]) {
    Pack<T, VE> o;
#pragma unroll
    for (int j = 0; j < VE; ++j) o.e[j] = from_f<T>(v[j]);
    o.put(p);
}

// Sum, or maximum of what is not negative, over the threads of a row: a warp, or the
// block.  `set` alternates from one of the block to the next: the barrier of each
// keeps the one before it apart from the one after.  Every thread has the same bits.
template <bool MAX = false>
__device__ __forceinline__ float row_sum(float v, int &set) {
    __shared__ float red[2][32];
    auto with = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = with(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (warps == 1) return v;
    if (lane == 0) red[set][threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? red[set][lane] : 0.f;
    set ^= 1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = with(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Threads of a block at most, by vectors per thread, and blocks on an SM: their
// registers.  Two vectors: three rows on an SM at a time.
constexpr int most_threads(int nv) { return nv == 1 ? 1024 : nv == 2 ? 384 : 512; }
constexpr int least_blocks(int nv) { return nv == 2 ? 3 : 1; }

// 1 / rms of D values whose squares' sum is ss, all of them times pre, as their root is.
__device__ __forceinline__ float inverse_rms(float ss, const BlockNorm &a, float pre = 1.f) {
    return rsqrtf(__fdividef(ss, (float)a.D) + a.eps * pre * pre);
}

// Whether f32 does not hold the squares of a row: their sum is past its largest number,
// or so small that single ones vanish (with an eps above 2^-100 they may).  Such a row
// is summed once more times a power of two; its largest magnitude tells which: it or
// sqrt(eps) comes near 2^40.  Not where it is 0 or infinite, nor for a NaN.
__device__ __forceinline__ bool out_of_range(float ss, const BlockNorm &a) {
    const float t = __fdividef(ss, (float)a.D) + a.eps;
    return t < 0x1p-100f || t > 0x1.fffffep127f;
}
__device__ __forceinline__ float factor_for(float top, const BlockNorm &a) {
    if (!(top > 0.f && top < INFINITY)) return 1.f;
    const int of_top = (int)(__float_as_uint(top) >> 23) - 127, of_eps = ((int)(__float_as_uint(a.eps) >> 23) - 127) >> 1;
    const int e = min(127, 40 - (a.eps > 0.f ? max(of_top, of_eps) : of_top));
    return __uint_as_float((unsigned)(127 + e) << 23);
}

// A thread's values: NV vectors of VE neighbours, the threads' next to each other,
// and where the vectors leave a row's first and last few out, one of those (a path
// of their own for the values of every partial vector is longer than all the rest,
// and code that is read from memory costs: 1571 x 6144 bf16 35.6 us with it).
// blockDim.y rows per block (more than one only where blockDim.x is one warp).
// SHIFT: row r begins r * ldm % VE values into a vector of the memory, in all operands.
template <class T, class Y, int VE, int NV, bool SHIFT>
__global__ void __launch_bounds__(most_threads(NV), least_blocks(NV)) block_norm_kernel(const __grid_constant__ BlockNorm a) {
    extern __shared__ float ws[];                // SHIFT: w_post, w and a gate for all rows, [3][VE][pitch]
    const int pitch = a.D / VE + 1, tid = threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // a gate for each value; a row of one column is one for the row
    const bool each = a.gate && a.gate_cols != 1, shared = SHIFT && each && a.ldg == 0;
    if constexpr (SHIFT) {
#pragma unroll 1
        for (int d = tid; d < a.D; d += blockDim.x) {
            const int to = d % VE * pitch + d / VE;
            if (a.w_post) ws[to] = a.w_post[d];
            if (a.y) ws[VE * pitch + to] = a.w[d];
            if (shared) ws[2 * VE * pitch + to] = to_f(((const T *)a.gate)[d]);
        }
        __syncthreads();
    }
    const long long step = (long long)gridDim.x * blockDim.y;
    long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    int set = 0;
    // Of a row: values before the first vector, vectors, this thread's single value (-1: none).
    int head = 0, nvec = a.D / VE, edge = -1;
    auto layout = [&](long long r) {
        if constexpr (SHIFT) {
            head = (VE - (int)(r * a.ldm & (VE - 1))) & (VE - 1);
            nvec = (a.D - head) / VE;
        }
        const int tail = head + nvec * VE;
        edge = tid < head ? tid : tid >= VE && tail + tid - VE < a.D ? tail + tid - VE : -1;
    };
    Pack<T, VE> mv[NV], hv[NV], gv[NV];
    T me, he, ge;
    auto fetch = [&]() {
        layout(row);
        const T *m = (const T *)a.m + row * a.ldm, *h = (const T *)a.h + row * a.ldh, *g = (const T *)a.gate + row * a.ldg;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = min(k * (int)blockDim.x + tid, nvec - 1);    // a vector past the last is read and not used
            mv[k].fetch(m + head + i * VE);
            if (a.h) hv[k].fetch(h + head + i * VE);
            if (each && !shared) gv[k].fetch(g + head + i * VE);
        }
        if (edge >= 0) {
            me = m[edge];
            if (a.h) he = h[edge];
            if (each && !shared) ge = g[edge];
        }
    };
    // the weights of vector i and of a single column
    auto weights = [&](const float *w, int which, int hd, int i) {
        Pack<float, VE> o;
        if constexpr (!SHIFT) {
            o.get(w + i * VE);
        } else {
#pragma unroll
            for (int j = 0; j < VE; ++j) o.e[j] = ws[(which * VE + ((hd + j) & (VE - 1))) * pitch + i + (hd + j >= VE ? 1 : 0)];
        }
        return o;
    };
    auto weight = [&](const float *w, int which, int c) { return SHIFT ? ws[(which * VE + c % VE) * pitch + c / VE] : w[c]; };
    if (row < a.S) fetch();
#pragma unroll 1
    for (; row < a.S;) {                         // whole warps; all of a block's where it has one row at a time
        const long long now = row;
        const int hd = head, nv = nvec, ed = edge;
        float scale = a.out_scale;
        if (a.gate && !each) scale *= to_f(((const T *)a.gate)[row * a.ldg]);
        if (a.w_post) {
            auto squares = [&]() {
                float ss = ed >= 0 ? to_f(me) * to_f(me) : 0.f;
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (k * (int)blockDim.x + tid < nv) {
#pragma unroll
                        for (int j = 0; j < VE; ++j) ss = fmaf(to_f(mv[k].e[j]), to_f(mv[k].e[j]), ss);
                    }
                return row_sum(ss, set);
            };
            float ss = squares(), pre = 1.f;
            if constexpr (!std::is_same<T, __half>::value) {               // f32 holds the squares of f16
                if (out_of_range(ss, a)) {
                    float top = ed >= 0 ? fabsf(to_f(me)) : 0.f;
#pragma unroll
                    for (int k = 0; k < NV; ++k)
                        if (k * (int)blockDim.x + tid < nv) {
#pragma unroll
                            for (int j = 0; j < VE; ++j) top = fmaxf(top, fabsf(to_f(mv[k].e[j])));
                        }
                    pre = factor_for(row_sum<true>(top, set), a);
                    if (ed >= 0) me = from_f<T>(to_f(me) * pre);           // exact, but for what is below the row's last place
#pragma unroll
                    for (int k = 0; k < NV; ++k)
#pragma unroll
                        for (int j = 0; j < VE; ++j) mv[k].e[j] = from_f<T>(to_f(mv[k].e[j]) * pre);
                    ss = squares();
                }
            }
            scale *= inverse_rms(ss, a, pre);
        }
        float v[NV][VE], ve = 0.f, ss = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = k * (int)blockDim.x + tid;
            if (i >= nv) continue;
#pragma unroll
            for (int j = 0; j < VE; ++j) v[k][j] = to_f(mv[k].e[j]) * scale;
            if (a.w_post) {
                const Pack<float, VE> w = weights(a.w_post, 0, hd, i);
#pragma unroll
                for (int j = 0; j < VE; ++j) v[k][j] *= w.e[j];
            }
            if (shared) {
                const Pack<float, VE> w = weights(nullptr, 2, hd, i);
#pragma unroll
                for (int j = 0; j < VE; ++j) v[k][j] *= w.e[j];
            } else if (each) {
#pragma unroll
                for (int j = 0; j < VE; ++j) v[k][j] *= to_f(gv[k].e[j]);
            }
            if (a.h) {
#pragma unroll
                for (int j = 0; j < VE; ++j) v[k][j] = fmaf(a.res_scale, to_f(hv[k].e[j]), v[k][j]);
            }
#pragma unroll
            for (int j = 0; j < VE; ++j) ss = fmaf(v[k][j], v[k][j], ss);
        }
        if (ed >= 0) {
            ve = to_f(me) * scale;
            if (a.w_post) ve *= weight(a.w_post, 0, ed);
            if (each) ve *= shared ? weight(nullptr, 2, ed) : to_f(ge);
            if (a.h) ve = fmaf(a.res_scale, to_f(he), ve);
            ss = fmaf(ve, ve, ss);
        }
        row += step;
        if (row < a.S) fetch();
        if (a.h_out) {
            T *o = (T *)a.h_out + now * a.ldo;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (k * (int)blockDim.x + tid < nv) store<T, VE>(o + hd + (k * (int)blockDim.x + tid) * VE, v[k]);
            if (ed >= 0) o[ed] = from_f<T>(ve);
        }
        if (a.y) {
            float pre = 1.f;
            ss = row_sum(ss, set);
            if (out_of_range(ss, a)) {
                float top = ed >= 0 ? fabsf(ve) : 0.f;
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (k * (int)blockDim.x + tid < nv) {
#pragma unroll
                        for (int j = 0; j < VE; ++j) top = fmaxf(top, fabsf(v[k][j]));
                    }
                pre = factor_for(row_sum<true>(top, set), a);
                ve *= pre;
                ss = ed >= 0 ? ve * ve : 0.f;
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (k * (int)blockDim.x + tid < nv) {
#pragma unroll
                        for (int j = 0; j < VE; ++j) v[k][j] *= pre, ss = fmaf(v[k][j], v[k][j], ss);
                    }
                ss = row_sum(ss, set);
            }
            const float root = inverse_rms(ss, a, pre);
            Y *y = (Y *)a.y + now * a.ldy;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int i = k * (int)blockDim.x + tid;
                if (i >= nv) continue;
                const Pack<float, VE> w = weights(a.w, 1, hd, i);
#pragma unroll
                for (int j = 0; j < VE; ++j) v[k][j] *= root * w.e[j];
                store<Y, VE>(y + hd + i * VE, v[k]);
            }
            if (ed >= 0) y[ed] = from_f<Y>(ve * (root * weight(a.w, 1, ed)));
        }
    }
}

// Rows longer than a block's registers hold: a block per row, each pass over the
// row from memory again.
constexpr int kLongThreads = 1024;

template <class T, class Y>
__global__ void __launch_bounds__(kLongThreads) block_norm_long_kernel(const __grid_constant__ BlockNorm a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long row = blockIdx.x;
    const T *m = (const T *)a.m + row * a.ldm;
    const T *h = a.h ? (const T *)a.h + row * a.ldh : nullptr;
    const T *g = a.gate ? (const T *)a.gate + row * a.ldg : nullptr;
    T *o = a.h_out ? (T *)a.h_out + row * a.ldo : nullptr;
    Y *y = a.y ? (Y *)a.y + row * a.ldy : nullptr;
    const unsigned D = a.D;                      // d passes 2^31 - 1 by up to a block
    // 1 / rms of the values of(d), times the power of two `pre` where f32 does not hold their squares
    int set = 0;
    auto root_of = [&](auto of, float &pre) {
        pre = 1.f;
        float ss = 0.f;
        for (unsigned d = threadIdx.x; d < D; d += kLongThreads) ss = fmaf(of(d), of(d), ss);
        ss = row_sum(ss, set);
        if (out_of_range(ss, a)) {
            float top = 0.f;
            for (unsigned d = threadIdx.x; d < D; d += kLongThreads) top = fmaxf(top, fabsf(of(d)));
            pre = factor_for(row_sum<true>(top, set), a);
            ss = 0.f;
            for (unsigned d = threadIdx.x; d < D; d += kLongThreads) ss = fmaf(of(d) * pre, of(d) * pre, ss);
            ss = row_sum(ss, set);
        }
        return inverse_rms(ss, a, pre);
    };
    float post = a.out_scale, pre_m = 1.f, pre_h = 1.f, root = 0.f;
    if (a.w_post) post *= root_of([&](unsigned d) { return to_f(m[d]); }, pre_m);
    auto next = [&](unsigned d) {
        float p = to_f(m[d]) * pre_m * post;
        if (a.w_post) p *= a.w_post[d];
        if (g) p *= to_f(g[a.gate_cols == 1 ? 0 : d]);
        return h ? fmaf(a.res_scale, to_f(h[d]), p) : p;
    };
    if (y) root = root_of(next, pre_h);
    for (unsigned d = threadIdx.x; d < D; d += kLongThreads) {
        const float v = next(d);                 // before this thread's write of h_out[d], which may be h or m
        if (o) o[d] = from_f<T>(v);
        if (y) y[d] = from_f<Y>(v * pre_h * (root * a.w[d]));
    }
}

template <class T, class Y, int VE, bool SHIFT>
cudaError_t start(const BlockNorm &a, cudaStream_t st) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int sms = sm_count(dev);
    const bool many = a.S > 2 * sms;
    const int units = a.D / VE < 1 ? 1 : a.D / VE;         // vectors of a row
    // few rows: as many threads as there are vectors, the shortest chain; many:
    // several vectors per thread, several blocks per SM
    int nv = 1;
    auto threads = [&](int n) { return ((units + n - 1) / n + 31) / 32 * 32; };
    while (nv < 4 && threads(nv) > (many && nv == 1 ? 128 : most_threads(nv))) nv *= 2;
    dim3 block(threads(nv));
    if ((int)block.x > most_threads(nv))
        return launch_dependent(block_norm_long_kernel<T, Y>, dim3(a.S), kLongThreads, 0, st, a);
    if (many && !SHIFT && units <= 128) {        // short rows: a warp each, eight to a block, no barrier
        nv = units <= 32 ? 1 : units <= 64 ? 2 : 4;
        block = dim3(32, 8);
    }
    const int size = (int)(block.x * block.y), fit = 65536 / ((nv == 1 ? 64 : nv == 2 ? 56 : 128) * size), on_sm = fit < 1 ? 1 : fit;
    const long long rows = (a.S + (long long)block.y - 1) / block.y;
    const dim3 grid((unsigned)(rows < (long long)on_sm * sms ? rows : (long long)on_sm * sms));
    const size_t smem = SHIFT ? (size_t)3 * VE * (a.D / VE + 1) * 4 : 0;
    auto go = [&](auto kernel) {
        if (smem > 40 * 1024) {                  // 48 KB in all without asking, the sums' own included
            cudaError_t r = allow_dynamic_smem((const void *)kernel, (int)smem);
            if (r != cudaSuccess) return r;
        }
        return launch_dependent(kernel, grid, block, smem, st, a);
    };
    if (nv == 1) return go(block_norm_kernel<T, Y, VE, 1, SHIFT>);
    if (nv == 2) return go(block_norm_kernel<T, Y, VE, 2, SHIFT>);
    return go(block_norm_kernel<T, Y, VE, 4, SHIFT>);
}

template <class T, class Y>
cudaError_t with_types(const BlockNorm &a, cudaStream_t st) {
    constexpr int VE = 16 / (int)sizeof(T), yb = VE * (int)sizeof(Y) < 16 ? VE * (int)sizeof(Y) : 16;
    const bool each = a.gate && a.gate_cols != 1;
    auto at = [](const void *p, int to) { return !p || (uintptr_t)p % to == 0; };
    const bool based = at(a.m, 16) && at(a.h, 16) && at(a.h_out, 16) && (!each || at(a.gate, 16)) && at(a.y, yb);
    auto alike = [&](const void *p, long long ld, long long to) { return !p || (ld - to) % VE == 0; };
    auto all = [&](long long to) {
        return alike(a.m, a.ldm, to) && alike(a.h, a.ldh, to) && alike(a.h_out, a.ldo, to) &&
               (!each || a.ldg == 0 || alike(a.gate, a.ldg, to)) && alike(a.y, a.ldy, to);
    };
    if (a.D < 2 * VE) return start<T, Y, 1, false>(a, st);      // a row has one whole vector at least
    if (based && all(0) && at(a.w_post, 16) && (!a.y || at(a.w, 16))) return start<T, Y, VE, false>(a, st);
    if (based && (all(a.ldm) || a.S == 1) && a.D <= 16384) return start<T, Y, VE, true>(a, st);
    return start<T, Y, 1, false>(a, st);
}

template <class T>
cudaError_t run(const BlockNorm &a, cudaStream_t st) {
    switch (a.y ? a.ytype : a.type) {
    case B200Q_T_F32: return with_types<T, float>(a, st);
    case B200Q_T_F16: return with_types<T, __half>(a, st);
    default: return with_types<T, __nv_bfloat16>(a, st);
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
