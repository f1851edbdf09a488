// 8-bit rows, few of them (S <= 8): matrix product and gated pair that stream
// the weights once at memory speed.
//     y[s,o] = act(scale[o] xs[s] sum_i deq(W[o,i]) x8[s,i] + bias[o]) + res[s,o],  or act(g) u
//
// Bound: HBM (the weights).  A weight costs an f32 FMA per row and an integer
// instruction or more on SIMT; here the products go to the warp-level tensor
// instruction m16n8k16 (f16 in, f32 sums): 16 weight rows against 8 tokens.
// The tcgen05 kernel needs 128 weight rows per tile, which leaves too few
// tiles to fill the GPU at one token without splitting K between CTAs.
//   * Codes and E4M3 values are exact in f16, so every product is exact.  An
//     int4 field ORed into the mantissa of 1024 is 1024 + c (or 1024 + 16 c,
//     one position up): one LOP3 and one packed f16 FMA per two weights.
//   * The order of K inside an instruction is free as long as both operands
//     agree: a thread keeps the order in which the fields of its own 16 bytes
//     of codes come apart, and x is stored in shared memory in that order.
//   * Weights go from global memory straight to registers, 16 bytes per thread
//     and row, several steps ahead; a warp's step is 64 bytes of 16 rows, and
//     the warps of a CTA take neighbouring steps of one tile, so K is split
//     over them and their sums are added in warp order at the end of the tile.
//   * The first steps' loads are issued before the dependency wait (the
//     weights are never written after their upload), and so run under the
//     previous kernel's end and the staging of x.
#include <cuda_fp16.h>

#include "qmat_q8.h"

namespace qwq {
namespace {

constexpr int kTokens = 8;
constexpr int kTileRows = 16;

// KC: codes in 16 bytes.  WORDS: mma instructions per 32-bit word of codes.
template <int FMT> struct Fmt;
template <> struct Fmt<B200Q_I8> { static constexpr int KC = 16, MMAS = 1; };
template <> struct Fmt<B200Q_I4> { static constexpr int KC = 32, MMAS = 2; };
template <> struct Fmt<B200Q_I2> { static constexpr int KC = 64, MMAS = 4; };

struct MvParams {
    const uint8_t *codes[2];
    const float *scale[2], *bias[2];
    const uint8_t *x8;
    const float *xs;
    const void *res;
    void *y;
    long long ld, ld8, ldr, ldy;
    int O, I, S, tiles, ng, act, type;      // ng: 64-byte groups of a row of codes
    int pitch;                              // bytes of a token's x in shared memory
};

__device__ __forceinline__ uint32_t lop_or(uint32_t w, uint32_t mask, uint32_t magic) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(magic));
    return r;
}

__device__ __forceinline__ uint32_t h2(uint32_t a, uint32_t mul, uint32_t add) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(mul), "r"(add));
    return r;
}

// A word of codes -> pairs of exact f16 values, pair 2 m and 2 m + 1 for
// instruction m.  f16 constants: 0x6400 = 1024; products and sums are exact.
template <int FMT>
__device__ __forceinline__ void pairs(uint32_t w, uint32_t (&p)[2 * Fmt<FMT>::MMAS]) {
    constexpr uint32_t k1024 = 0x64006400u, one = 0x3C003C00u;
    if constexpr (FMT == B200Q_I8) {                      // natural order: 1024 + (c + 128) - 1152
        const uint32_t u = w ^ 0x80808080u;
        p[0] = h2(__byte_perm(u, k1024, 0x5150), one, 0xE480E480u);
        p[1] = h2(__byte_perm(u, k1024, 0x5352), one, 0xE480E480u);
    } else if constexpr (FMT == B200Q_I4) {               // (0,4) (1,5) (2,6) (3,7)
        const uint32_t v = w >> 8;
        p[0] = h2(lop_or(w, 0x000F000Fu, k1024), one, 0xE408E408u);            // - 1032
        p[1] = h2(lop_or(w, 0x00F000F0u, k1024), 0x2C002C00u, 0xD480D480u);    // / 16 - 72
        p[2] = h2(lop_or(v, 0x000F000Fu, k1024), one, 0xE408E408u);
        p[3] = h2(lop_or(v, 0x00F000F0u, k1024), 0x2C002C00u, 0xD480D480u);
    } else {                                              // (0,8) (1,9) .. (7,15)
        const uint32_t v = w >> 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t q = h ? v : w;
            p[4 * h] = h2(lop_or(q, 0x00030003u, k1024), one, 0xE402E402u);                // - 1026
            p[4 * h + 1] = h2(lop_or(q, 0x000C000Cu, k1024), 0x34003400u, 0xDC08DC08u);    // / 4 - 258
            p[4 * h + 2] = h2(lop_or(q, 0x00300030u, k1024), 0x2C002C00u, 0xD420D420u);    // / 16 - 66
            p[4 * h + 3] = h2(lop_or(q, 0x00C000C0u, k1024), 0x24002400u, 0xCC80CC80u);    // / 64 - 18
        }
    }
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_codes(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Two E4M3 bytes -> two f16 (exact).
__device__ __forceinline__ uint32_t e4m3_h2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
    return r;
}

// 16 bytes of x8 (columns k0 ..) into a token's staged row.
template <int FMT>
__device__ __forceinline__ void stage16(uint8_t *row, int k0, uint4 q) {
    constexpr int KC = Fmt<FMT>::KC;
    const uint32_t b[4] = {q.x, q.y, q.z, q.w};
    uint32_t n[8];                                     // natural pairs (0,1) (2,3) ..
#pragma unroll
    for (int i = 0; i < 4; ++i) n[2 * i] = e4m3_h2(b[i] & 0xFFFFu), n[2 * i + 1] = e4m3_h2(b[i] >> 16);
    const int c = k0 / KC, tig = c & 3, grp = c >> 2;
    uint8_t *dst = row + (size_t)grp * (8 * KC) + tig * 16 + (k0 % KC) / 8 * 64;
    uint4 lo, hi;
    if constexpr (FMT == B200Q_I8) {
        lo = make_uint4(n[0], n[1], n[2], n[3]);
        hi = make_uint4(n[4], n[5], n[6], n[7]);
    } else if constexpr (FMT == B200Q_I4) {            // each eight as (0,4) (1,5) (2,6) (3,7)
        lo = make_uint4(__byte_perm(n[0], n[2], 0x5410), __byte_perm(n[0], n[2], 0x7632),
                        __byte_perm(n[1], n[3], 0x5410), __byte_perm(n[1], n[3], 0x7632));
        hi = make_uint4(__byte_perm(n[4], n[6], 0x5410), __byte_perm(n[4], n[6], 0x7632),
                        __byte_perm(n[5], n[7], 0x5410), __byte_perm(n[5], n[7], 0x7632));
    } else {                                           // sixteen as (0,8) (1,9) .. (7,15)
        lo = make_uint4(__byte_perm(n[0], n[4], 0x5410), __byte_perm(n[0], n[4], 0x7632),
                        __byte_perm(n[1], n[5], 0x5410), __byte_perm(n[1], n[5], 0x7632));
        hi = make_uint4(__byte_perm(n[2], n[6], 0x5410), __byte_perm(n[2], n[6], 0x7632),
                        __byte_perm(n[3], n[7], 0x5410), __byte_perm(n[3], n[7], 0x7632));
    }
    *reinterpret_cast<uint4 *>(dst) = lo;
    *reinterpret_cast<uint4 *>(dst + 64) = hi;
}

template <int FMT, bool GLU>
__global__ void __launch_bounds__(1024, 1) qmv_q8_kernel(const MvParams p) {
    constexpr int KC = Fmt<FMT>::KC, MMAS = Fmt<FMT>::MMAS, M = GLU ? 2 : 1;
    constexpr int kAhead = GLU ? 2 : 4;                // steps in flight per warp
    extern __shared__ __align__(128) uint8_t smem[];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, tig = lane & 3;
    float *red = reinterpret_cast<float *>(smem + (size_t)p.S * p.pitch);      // [warps][M][128]
    const int steps = p.ng > warp ? (p.ng - warp + warps - 1) / warps : 0;     // of this warp per tile

    uint4 q[kAhead][M][2];
    const uint8_t *src[M];
    auto aim = [&](int tile) {
#pragma unroll
        for (int m = 0; m < M; ++m)
            src[m] = p.codes[m] + ((long long)tile * kTileRows + g) * p.ld + warp * 64 + tig * 16;
    };
    auto fetch = [&](int slot, int st) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            q[slot][m][0] = load_codes(src[m] + (long long)st * warps * 64);
            q[slot][m][1] = load_codes(src[m] + (long long)st * warps * 64 + 8 * p.ld);
        }
    };
    aim(blockIdx.x);
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
        if (s < steps) fetch(s, s);

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // x, in f16 and the codes' order, zero past I
    const int kpad = p.ng * 4 * KC;
    for (int s = 0; s < p.S; ++s) {
        const uint8_t *xr = p.x8 + s * p.ld8;
        uint8_t *row = smem + (size_t)s * p.pitch;
        for (int k = threadIdx.x * 16; k < kpad; k += blockDim.x * 16) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (k + 16 <= p.I) {
                v = *reinterpret_cast<const uint4 *>(xr + k);
            } else if (k < p.I) {
                uint32_t w[4] = {0u, 0u, 0u, 0u};
                for (int j = 0; k + j < p.I; ++j) w[j >> 2] |= (uint32_t)xr[k + j] << (8 * (j & 3));
                v = make_uint4(w[0], w[1], w[2], w[3]);
            }
            stage16<FMT>(row, k, v);
        }
    }
    __syncthreads();

    const bool have = g < p.S;
    const uint8_t *xb = smem + (size_t)(have ? g : 0) * p.pitch + tig * 16 + (size_t)warp * (8 * KC);
    for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        float acc[M][4] = {};
        for (int s0 = 0; s0 < steps; s0 += kAhead) {
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int st = s0 + a;
                if (st >= steps) break;
                const uint8_t *xp = xb + (size_t)st * warps * (8 * KC);
#pragma unroll
                for (int i = 0; i < 4; ++i) {           // words of the 16 bytes
                    uint32_t b[2 * MMAS];
                    if constexpr (MMAS == 1) {
                        uint2 v = make_uint2(0u, 0u);
                        if (have) v = *reinterpret_cast<const uint2 *>(xp + (i >> 1) * 64 + (i & 1) * 8);
                        b[0] = v.x, b[1] = v.y;
                    } else {
#pragma unroll
                        for (int h = 0; h < MMAS / 2; ++h) {
                            uint4 v = make_uint4(0u, 0u, 0u, 0u);
                            if (have) v = *reinterpret_cast<const uint4 *>(xp + (i * (MMAS / 2) + h) * 64);
                            b[4 * h] = v.x, b[4 * h + 1] = v.y, b[4 * h + 2] = v.z, b[4 * h + 3] = v.w;
                        }
                    }
#pragma unroll
                    for (int m = 0; m < M; ++m) {
                        uint32_t lo[2 * MMAS], hi[2 * MMAS];
                        const uint4 &c0 = q[a][m][0], &c1 = q[a][m][1];
                        pairs<FMT>(i == 0 ? c0.x : i == 1 ? c0.y : i == 2 ? c0.z : c0.w, lo);
                        pairs<FMT>(i == 0 ? c1.x : i == 1 ? c1.y : i == 2 ? c1.z : c1.w, hi);
#pragma unroll
                        for (int t = 0; t < MMAS; ++t)
                            mma_f16(acc[m], lo[2 * t], hi[2 * t], lo[2 * t + 1], hi[2 * t + 1], b[2 * t], b[2 * t + 1]);
                    }
                }
                if (st + kAhead < steps) fetch(a, st + kAhead);
            }
        }
        const int next = tile + gridDim.x;
        if (next < p.tiles) {
            aim(next);
#pragma unroll
            for (int s = 0; s < kAhead; ++s)
                if (s < steps) fetch(s, s);
        }
        // [row][token] of the tile, added over the warps in order
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float *r = red + (warp * M + m) * 128;
            *reinterpret_cast<float2 *>(r + g * 8 + 2 * tig) = make_float2(acc[m][0], acc[m][1]);
            *reinterpret_cast<float2 *>(r + (g + 8) * 8 + 2 * tig) = make_float2(acc[m][2], acc[m][3]);
        }
        __syncthreads();
        for (int e = threadIdx.x; e < 128; e += blockDim.x) {
            const int s = e >> 4, r = e & 15, o = tile * kTileRows + r;
            if (s >= p.S || o >= p.O) continue;
            float v[M];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                float sum = 0.f;
                for (int w = 0; w < warps; ++w) sum += red[(w * M + m) * 128 + r * 8 + s];
                v[m] = fmaf(sum, p.xs[s] * p.scale[m][o], p.bias[m] ? p.bias[m][o] : 0.f);
            }
            float out = act_q8(v[0], p.act);
            if constexpr (GLU) out *= v[1];
            if (p.res) out += load_typed(p.res, s * p.ldr + o, p.type);
            store_typed(p.y, s * p.ldy + o, p.type, out);
        }
        __syncthreads();
    }
}

template <int FMT, bool GLU>
cudaError_t run(const MatQ8 &a, cudaStream_t st, bool *handled) {
    constexpr int KC = Fmt<FMT>::KC, M = GLU ? 2 : 1;
    const Tensor &t = *a.tg;
    MvParams p{};
    p.codes[0] = t.codes;
    p.scale[0] = t.scales;
    p.bias[0] = a.bias_g;
    p.codes[1] = GLU ? a.tu->codes : nullptr;
    p.scale[1] = GLU ? a.tu->scales : nullptr;
    p.bias[1] = a.bias_u;
    p.x8 = a.x8;
    p.xs = a.xs;
    p.res = a.res;
    p.y = a.y;
    p.ld = t.ld;
    p.ld8 = a.ld8;
    p.ldr = a.ldr;
    p.ldy = a.ldy;
    p.O = t.O;
    p.I = t.I;
    p.S = a.S;
    p.tiles = (t.O + kTileRows - 1) / kTileRows;
    p.ng = (int)(t.ld / 64);
    p.act = a.act;
    p.type = a.type;
    p.pitch = p.ng * 8 * KC + 64;                       // 64 bytes off a 128-byte multiple: two tokens' reads differ in bank
    // 32 warps per SM: four CTAs of 8, two of 16 or one of 32, as x fits
    const long long xbytes = (long long)a.S * p.pitch;
    int warps = 8;
    while (warps <= 32 && (xbytes + (long long)warps * M * 512 + 1024) * (32 / warps) > 228 * 1024) warps *= 2;
    if (warps > 32) return cudaSuccess;                 // x does not fit: not handled here
    const size_t smem = (size_t)xbytes + (size_t)warps * M * 512;
    cudaError_t e = allow_dynamic_smem((const void *)qmv_q8_kernel<FMT, GLU>, 227 * 1024);
    if (e != cudaSuccess) return e;
    const int slots = sm_count(t.device) * (32 / warps);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.tiles < slots ? p.tiles : slots);
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, qmv_q8_kernel<FMT, GLU>, p);
    count_launch();
    *handled = true;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// S <= 8; *handled = false where x does not fit in shared memory.
cudaError_t launch_mv_q8(const MatQ8 &a, cudaStream_t st, bool *handled) {
    *handled = false;
    if (a.S > kTokens) return cudaSuccess;
    switch (a.tg->fmt) {
    case B200Q_I8: return a.tu ? run<B200Q_I8, true>(a, st, handled) : run<B200Q_I8, false>(a, st, handled);
    case B200Q_I4: return a.tu ? run<B200Q_I4, true>(a, st, handled) : run<B200Q_I4, false>(a, st, handled);
    case B200Q_I2: return a.tu ? run<B200Q_I2, true>(a, st, handled) : run<B200Q_I2, false>(a, st, handled);
    }
    return cudaErrorInvalidValue;
}

}  // namespace qwq
