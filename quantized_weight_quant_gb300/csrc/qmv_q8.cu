// 8-bit rows, few of them (S <= 8): matrix product and gated pair that stream
// the weights once at memory speed.
//     y[s,o] = act(scale[o] xs[s] sum_i deq(W[o,i]) x8[s,i] + bias[o]) + res[s,o],  or act(g) u
//
// Bound: HBM (the weights); now a call's start and the integer work on the
// codes: int4 6144 x 12288, one token, 12.0 us, 3150 GB/s; the 12288 x 6144 pair
// 19.7 us, 3830 GB/s; int8 8192 x 8192, 8 tokens, 17.6 us, 3810 GB/s.  A weight costs an f32 FMA per row and an integer
// instruction or more on SIMT; here the products go to the warp-level tensor
// instruction m16n8k16 (f16 in, f32 sums): 16 weight rows against 8 tokens.
// The tcgen05 kernel needs 128 weight rows per tile, which leaves too few
// tiles to fill the GPU at one token without splitting K between CTAs.
//   * Codes (signed) and E4M3 values are exact in f16, so every product is
//     exact; sums are f32.  An int4 field ORed into the mantissa of 1024 is
//     1024 + c (or 1024 + 16 c, one position up): one LOP3 and one packed f16
//     FMA per two weights.  (Unsigned fields as f16 subnormals, with the zero
//     point times sum_i x8 taken off at the end, need no FMA, but lose the
//     bound where a large x meets codes that stand for zero.  The E4M3 form of
//     the instruction costs more: its operands are widened first.)
//   * The order of K inside an instruction is free as long as both operands
//     agree: a thread keeps the order in which the fields of its own 16 bytes
//     of codes come apart, and x is stored in shared memory in that order.
//   * x is staged in f16 where that leaves room for the ring, otherwise as its
//     bytes, which become f16 in registers.
//   * Each thread copies its own 16 bytes of codes per row and step to its own
//     slot of a ring in shared memory (cp.async), several steps ahead and
//     across tile boundaries; nothing but its own wait orders them.  A warp's
//     step is 64 bytes of 16 rows; the warps of a CTA take neighbouring steps
//     of one tile, so K is split over them and their sums are added in warp
//     order at the end of the tile.
//   * The ring is filled before the dependency wait (the weights are never
//     written after their upload): memory works under the previous kernel's
//     end and the staging of x.  How much of that end depends on when the
//     previous kernel lets this one start: a kernel like this one does at once,
//     the row kernels and the tcgen05 one only as their blocks exit (norm, pair,
//     rows, product of 6144 / 12288 int4, one token: 42.6 us in a graph, the four
//     repeated each by itself 40.3 us).
#include <cuda_fp16.h>

#include "codes_f16.h"
#include "qmat_q8.h"

namespace qwq {
namespace {

constexpr int kTokens = 8;
constexpr int kTileRows = 16;

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

// 16 bytes of x8 in the order of fields(): word h holds the two pairs of
// instruction h % MMAS.
template <int FMT>
__device__ __forceinline__ uint4 permuted(uint4 q) {
    if constexpr (FMT == B200Q_I8) return q;
    if constexpr (FMT == B200Q_I4)
        return make_uint4(__byte_perm(q.x, q.y, 0x6240), __byte_perm(q.x, q.y, 0x7351), __byte_perm(q.z, q.w, 0x6240),
                          __byte_perm(q.z, q.w, 0x7351));
    const uint32_t a = __byte_perm(q.x, q.z, 0x5140), b = __byte_perm(q.y, q.w, 0x5140);
    const uint32_t c = __byte_perm(q.x, q.z, 0x7362), d = __byte_perm(q.y, q.w, 0x7362);
    return make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632), __byte_perm(c, d, 0x5410),
                      __byte_perm(c, d, 0x7632));
}

// Two E4M3 bytes -> two f16 (exact).
__device__ __forceinline__ uint32_t x_pair(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
    return r;
}

// 16 bytes of x8 (columns k0 ..) into a token's staged row: per 64-byte group
// of codes, the 16-byte pieces of its four chunks side by side.
template <int FMT, bool XH>
__device__ __forceinline__ void stage16(uint8_t *row, int k0, uint4 q) {
    constexpr int KC = Fmt<FMT>::KC;
    const int c = k0 / KC, tig = c & 3, grp = c >> 2, in = (k0 % KC) / 16;
    if constexpr (!XH) {
        *reinterpret_cast<uint4 *>(row + grp * (4 * KC) + in * 64 + tig * 16) = q;
    } else {
        uint8_t *dst = row + grp * (8 * KC) + in * 128 + tig * 16;
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        uint32_t f[8];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            f[2 * h] = x_pair(w[h] & 0xFFFFu);
            f[2 * h + 1] = x_pair(w[h] >> 16);
        }
        *reinterpret_cast<uint4 *>(dst) = make_uint4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<uint4 *>(dst + 64) = make_uint4(f[4], f[5], f[6], f[7]);
    }
}

// AHEAD: steps in the ring.  XH: x staged in f16.
template <int FMT, bool GLU, bool XH, int AHEAD>
__global__ void __launch_bounds__(1024, 1) qmv_q8_kernel(const MvParams p) {
    constexpr int KC = Fmt<FMT>::KC, MMAS = Fmt<FMT>::MMAS, M = GLU ? 2 : 1;
    constexpr int kGroup = (XH ? 8 : 4) * KC;          // bytes of a token's x per 64-byte group of codes
    constexpr int kSlot = M * 1024;                    // bytes of a warp's step: [M][2 row halves][32 lanes] x 16
    extern __shared__ __align__(128) uint8_t smem[];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, tig = lane & 3;
    uint8_t *ring = smem + warp * (AHEAD * kSlot) + lane * 16;
    float *red = reinterpret_cast<float *>(smem + warps * (AHEAD * kSlot));     // [1 or 2][warps][M][128]
    uint8_t *xsm = smem + warps * (AHEAD * kSlot + (p.tiles <= (int)gridDim.x ? 1 : 2) * M * 512);
    const int steps = p.ng > warp ? (p.ng - warp + warps - 1) / warps : 0;      // of this warp per tile

    // the copy cursor runs AHEAD steps before the arithmetic
    int ftile = steps ? (int)blockIdx.x : p.tiles, fst = 0, fslot = 0;
    const uint32_t ring32 = (uint32_t)__cvta_generic_to_shared(ring);
    const long long tile_step = (long long)gridDim.x * kTileRows * p.ld - (long long)steps * warps * 64;
    const long long row8 = 8 * p.ld;
    long long off = ((long long)blockIdx.x * kTileRows + g) * p.ld + warp * 64 + tig * 16;
    auto copy_step = [&]() {
        if (ftile < p.tiles) {
#pragma unroll
            for (int m = 0; m < M; ++m) {
                copy16(ring32 + fslot * kSlot + m * 1024, p.codes[m] + off);
                copy16(ring32 + fslot * kSlot + m * 1024 + 512, p.codes[m] + off + row8);
            }
            off += warps * 64;
            if (++fst == steps) fst = 0, ftile += gridDim.x, off += tile_step;
            if (++fslot == AHEAD) fslot = 0;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");       // empty at the end: the waits count groups
    };
#pragma unroll 1
    for (int s = 0; s < AHEAD; ++s) copy_step();

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // x, zero past I
    const int cols = p.ng * 4 * KC;
    for (int s = 0; s < p.S; ++s) {
        const uint8_t *xr = p.x8 + s * p.ld8;
        uint8_t *row = xsm + s * p.pitch;
#pragma unroll 2
        for (int k = threadIdx.x * 16; k < cols; k += blockDim.x * 16) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (k + 16 <= p.I) {
                v = *reinterpret_cast<const uint4 *>(xr + k);
            } else if (k < p.I) {
                uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int j = 0; j < 15; ++j)
                    if (k + j < p.I) w[j >> 2] |= (uint32_t)xr[k + j] << (8 * (j & 3));
                v = make_uint4(w[0], w[1], w[2], w[3]);
            }
            stage16<FMT, XH>(row, k, permuted<FMT>(v));
        }
    }
    __syncthreads();

    const bool have = g < p.S;
    const uint8_t *xb = xsm + (have ? g : 0) * p.pitch + tig * 16 + warp * kGroup;
    int slot = 0, buf = 0;
    for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x, buf ^= 1) {
        float acc[M][4] = {};
        const uint8_t *xp = xb;
        for (int st = 0; st < steps; ++st, xp += warps * kGroup) {
            asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
            uint4 q[M][2];
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    q[m][h] = *reinterpret_cast<const uint4 *>(ring + slot * kSlot + m * 1024 + h * 512);
            if (++slot == AHEAD) slot = 0;
            constexpr int L = kGroup / 64;              // 16-byte pieces of x per chunk
            uint4 xv[L];
#pragma unroll
            for (int l = 0; l < L; ++l)
                xv[l] = have ? *reinterpret_cast<const uint4 *>(xp + l * 64) : make_uint4(0u, 0u, 0u, 0u);
            copy_step();       // into the slot just read: this thread's own, so no barrier
#pragma unroll
            for (int n = 0; n < 4 * MMAS; ++n) {
                const int i = n / MMAS, t = n % MMAS;   // word of the 16 bytes, instruction of the word
                uint32_t b0, b1;
                if constexpr (XH) {
                    const uint4 &v = xv[n / 2];
                    b0 = n & 1 ? v.z : v.x, b1 = n & 1 ? v.w : v.y;
                } else {
                    const uint4 &v = xv[n / 4];
                    const uint32_t e = n % 4 == 0 ? v.x : n % 4 == 1 ? v.y : n % 4 == 2 ? v.z : v.w;
                    b0 = x_pair(e & 0xFFFFu), b1 = x_pair(e >> 16);
                }
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const uint4 &c0 = q[m][0], &c1 = q[m][1];
                    uint32_t a0, a1, a2, a3;
                    fields<FMT>(i == 0 ? c0.x : i == 1 ? c0.y : i == 2 ? c0.z : c0.w, t, a0, a2);
                    fields<FMT>(i == 0 ? c1.x : i == 1 ? c1.y : i == 2 ? c1.z : c1.w, t, a1, a3);
                    mma_f16(acc[m], a0, a1, a2, a3, b0, b1);
                }
            }
        }
        // [row][token] of the tile, added over the warps in order; the two
        // buffers take turns, so that one barrier per tile is enough
        float *rb = red + buf * warps * M * 128;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float *r = rb + (warp * M + m) * 128;
            *reinterpret_cast<float2 *>(r + g * 8 + 2 * tig) = make_float2(acc[m][0], acc[m][1]);
            *reinterpret_cast<float2 *>(r + (g + 8) * 8 + 2 * tig) = make_float2(acc[m][2], acc[m][3]);
        }
        __syncthreads();
        if (threadIdx.x < 128) {
            const int s = threadIdx.x >> 4, r = threadIdx.x & 15, o = tile * kTileRows + r;
            if (s < p.S && o < p.O) {
                float v[M];
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    float sum = 0.f;
#pragma unroll 8
                    for (int w = 0; w < warps; ++w) sum += rb[(w * M + m) * 128 + r * 8 + s];
                    v[m] = fmaf(sum, p.xs[s] * p.scale[m][o], p.bias[m] ? p.bias[m][o] : 0.f);
                }
                float out = act_q8(v[0], p.act);
                if constexpr (GLU) out *= v[1];
                if (p.res) out += load_typed(p.res, s * p.ldr + o, p.type);
                store_typed(p.y, s * p.ldy + o, p.type, out);
            }
        }
    }
}

// Shared memory beside x and the ring: the warps' sums, two sets if a CTA takes
// more than one tile.
constexpr long long sums_bytes(int warps, int M, bool one) { return (long long)warps * (one ? 1 : 2) * M * 512; }

// CTAs per SM and warps per CTA.  First choice: every tile has its CTA from
// the start (up to eight CTAs of an SM's 32 warps), so that no CTA takes a
// second tile while others have none (6144 x 12288 int4, 384 tiles, one
// token: 12.0 us with 3 x 10 warps, 13.7 us with 2 x 16 and 304 of the 384
// tiles in the first round).  Otherwise 32 warps in a few CTAs that walk
// the tiles, 16 where x leaves no room for more.  x in f16 if it fits
// beside a ring of four steps (two of the pair) with two CTAs per SM or
// more, as bytes otherwise (12288 x 6144 int4, 8 tokens: f16 with one CTA
// 16.1 us, bytes with two 14.9 us).  Rows are 64 bytes off a 128-byte
// multiple: two tokens' reads differ in bank.
template <int FMT, bool GLU>
MvPlan plan(int O, long long ld, int S, int n_sms) {
    constexpr int KC = Fmt<FMT>::KC, M = GLU ? 2 : 1;
    MvPlan r{};
    r.tiles = (int)((O + (kTileRows - 1ll)) / kTileRows);
    r.ng = (int)(ld / 64);
    const int each = (int)((r.tiles + (n_sms - 1ll)) / n_sms);
    const int most = 32 / (each < 8 ? each : 8), steps = (r.ng + most - 1) / most;
    const int shapes[5][2] = {{each, (r.ng + steps - 1) / steps}, {4, 8}, {2, 16}, {1, 32}, {1, 16}};
    for (int xh = 1; xh >= 0; --xh)
        for (int k = each <= 8 ? 0 : 1; k < 5; ++k) {
            const int c = shapes[k][0], warps = shapes[k][1] < 4 ? 4 : shapes[k][1];     // four finish a tile
            const long long pitch = (long long)r.ng * (xh ? 8 : 4) * KC + 64;      // past 2^31 for the longest rows
            const long long sums = sums_bytes(warps, M, r.tiles <= n_sms * c);
            const long long room = 228 * 1024 / c - 1024 - S * pitch - sums;
            const long long ahead = room / (warps * M * 1024);
            if (ahead >= (GLU || !xh ? 2 : 4) && !(xh && c == 1 && k)) {
                r.fits = true;
                r.xh = xh;
                r.ahead = ahead >= 4 ? 4 : 2;
                r.warps = warps;
                r.pitch = (int)pitch;
                r.grid = r.tiles < n_sms * c ? r.tiles : n_sms * c;
                r.smem = S * pitch + sums + (long long)warps * M * r.ahead * 1024;
                return r;
            }
        }
    return r;                                           // x does not fit
}

template <int FMT, bool GLU, bool XH, int AHEAD>
cudaError_t start(const MvParams &p, const MvPlan &r, cudaStream_t st) {
    cudaError_t e = allow_dynamic_smem((const void *)qmv_q8_kernel<FMT, GLU, XH, AHEAD>, 227 * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(r.grid);
    cfg.blockDim = dim3(r.warps * 32);
    cfg.dynamicSmemBytes = (size_t)r.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, qmv_q8_kernel<FMT, GLU, XH, AHEAD>, p);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int FMT, bool GLU>
cudaError_t run(const MatQ8 &a, cudaStream_t st, bool *handled) {
    const Tensor &t = *a.tg;
    const MvPlan r = plan<FMT, GLU>(t.O, t.ld, a.S, sm_count(t.device));
    if (!r.fits) return cudaSuccess;
    *handled = true;
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
    p.tiles = r.tiles;
    p.ng = r.ng;
    p.act = a.act;
    p.type = a.type;
    p.pitch = r.pitch;
    if (r.xh) return r.ahead == 4 ? start<FMT, GLU, true, 4>(p, r, st) : start<FMT, GLU, true, 2>(p, r, st);
    return r.ahead == 4 ? start<FMT, GLU, false, 4>(p, r, st) : start<FMT, GLU, false, 2>(p, r, st);
}

}  // namespace

MvPlan plan_mv_q8(int fmt, bool pair, int O, long long ld, int S, int n_sms) {
    if (S > kTokens) return MvPlan{};
    switch (fmt) {
    case B200Q_I8: return pair ? plan<B200Q_I8, true>(O, ld, S, n_sms) : plan<B200Q_I8, false>(O, ld, S, n_sms);
    case B200Q_I4: return pair ? plan<B200Q_I4, true>(O, ld, S, n_sms) : plan<B200Q_I4, false>(O, ld, S, n_sms);
    case B200Q_I2: return pair ? plan<B200Q_I2, true>(O, ld, S, n_sms) : plan<B200Q_I2, false>(O, ld, S, n_sms);
    }
    return MvPlan{};
}

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
