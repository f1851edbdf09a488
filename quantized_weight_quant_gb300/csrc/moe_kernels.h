// Kernels of the experts' layer (moe_experts.cu has the overview): the plan that
// every block makes from the ids, and the products of each expert's matrices with
// its columns.  One translation unit per format instantiates them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "codes_f16.h"
#include "moe.h"
#include "qmat_q8.h"

namespace qwq {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRedPitch = 20;                 // floats of a column's 16 sums in shared memory: no bank conflicts

__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_dependents_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Codes pass through L2 once: they go first when room is needed, so that what a
// call reads again (activations, and the kernels' own instructions) stays.
__device__ __forceinline__ uint64_t stream_policy() {
    uint64_t r;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(r));
    return r;
}
__device__ __forceinline__ void prefetch(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ---------------------------------------------------------------- plan
// The slots in the order of their experts, in chunks of at most nc columns.
struct Plan {
    unsigned short order[kMoePairs];          // slots, by expert
    unsigned short expert[kMoePairs], first[kMoePairs];   // of chunk c: its expert, its first place in order
    unsigned char n[kMoePairs];               // and its columns
    int chunks;
};
struct PlanScratch {
    int count[kMoeMaxExperts];                // slots of an expert, then their first place
    unsigned short rank[kMoePairs];           // of a slot among its expert's
    short id[kMoePairs];
};

// Ends with a barrier.
__device__ __forceinline__ void make_plan(const MoeStream &p, Plan &pl, PlanScratch &sc) {
    const int tid = threadIdx.x, lane = tid & 31;
    auto expert_of = [&](int i) {
        const int e = p.ids[i];
        if (e >= 0 && e < p.E) return e;
        if (e != -1 && !p.down && blockIdx.x == 0) atomicCAS(p.err, 0u, (unsigned)(-B200Q_EINVAL));
        return -1;
    };
    if (p.P <= 32) {                           // one warp, no scratch
        if (tid < 32) {
            const int e = lane < p.P ? expert_of(lane) : -1;
            const unsigned same = __match_any_sync(kAll, e);
            const int c = __popc(same), rank = __popc(same & ((1u << lane) - 1)), m = e >= 0 && rank == 0 ? (c + p.nc - 1) / p.nc : 0;
            int place = 0, chunk = 0;          // slots and chunks of lower experts
            for (int t = 0; t < p.P; ++t) {
                const int et = __shfl_sync(kAll, e, t), mt = __shfl_sync(kAll, m, t);
                if (et >= 0 && et < e) ++place, chunk += mt;
            }
            if (e >= 0) pl.order[place + rank] = (unsigned short)lane;
            for (int j = 0; j < m; ++j) {
                pl.expert[chunk + j] = (unsigned short)e;
                pl.first[chunk + j] = (unsigned short)(place + j * p.nc);
                pl.n[chunk + j] = (unsigned char)min(p.nc, c - j * p.nc);
            }
            const int chunks = __reduce_add_sync(kAll, m);
            if (lane == 0) pl.chunks = chunks;
        }
        __syncthreads();
        return;
    }
    for (int e = tid; e < p.E; e += blockDim.x) sc.count[e] = 0;
    for (int i = tid; i < p.P; i += blockDim.x) sc.id[i] = (short)expert_of(i);
    __syncthreads();
    if (tid < 32) {
        // ranks in the order of the slots
        for (int i0 = 0; i0 < p.P; i0 += 32) {
            const int i = i0 + lane, e = i < p.P ? sc.id[i] : -1;
            const unsigned same = __match_any_sync(kAll, e);
            const int before = e >= 0 ? sc.count[e] : 0;
            __syncwarp();
            if (e >= 0) {
                sc.rank[i] = (unsigned short)(before + __popc(same & ((1u << lane) - 1)));
                if (lane == __ffs(same) - 1) sc.count[e] = before + __popc(same);
            }
            __syncwarp();
        }
        // first places and chunks
        int place = 0, chunk = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane, c = e < p.E ? sc.count[e] : 0, m = (c + p.nc - 1) / p.nc;
            int a = c, b = m;                  // sums up to and with this lane's
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int va = __shfl_up_sync(kAll, a, o), vb = __shfl_up_sync(kAll, b, o);
                if (lane >= o) a += va, b += vb;
            }
            const int f = place + a - c;
            if (e < p.E) sc.count[e] = f;
            for (int j = 0; j < m; ++j) {
                const int at = chunk + b - m + j;
                pl.expert[at] = (unsigned short)e;
                pl.first[at] = (unsigned short)(f + j * p.nc);
                pl.n[at] = (unsigned char)min(p.nc, c - j * p.nc);
            }
            place += __shfl_sync(kAll, a, 31);
            chunk += __shfl_sync(kAll, b, 31);
        }
        if (lane == 0) pl.chunks = chunk;
    }
    __syncthreads();
    for (int i = tid; i < p.P; i += blockDim.x)
        if (sc.id[i] >= 0) pl.order[sc.count[sc.id[i]] + sc.rank[i]] = (unsigned short)i;
    __syncthreads();
}

// ---------------------------------------------------------------- columns
// What runs once per block is kept small: its instructions come from memory, and
// that is most of what they cost (columns staged by code with every type and
// alignment inlined and unrolled: 8 us a product, this 1 us).

template <class T> __device__ __forceinline__ float as_float(T v);
template <> __device__ __forceinline__ float as_float<float>(float v) { return v; }
template <> __device__ __forceinline__ float as_float<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float as_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Where a product's columns come from: eight values of row `row` from c on, 0
// from K on.  kTop: what the exponent of a column's largest value is brought to,
// 15 where rounding to f16 cannot carry it past 65504.  The tokens' rows:
template <class T> struct TokenRows {
    static constexpr int kTop = sizeof(T) == 2 ? 15 : 14;
    static __device__ __forceinline__ const T *at(const MoeStream &p, int row, int c) { return (const T *)p.x + row * p.ldx + c; }
    static __device__ __forceinline__ void load(const MoeStream &p, int row, int c, float (&v)[8]) {
        const T *r = at(p, row, c);
        if (p.aligned && c + 8 <= p.K) {
            union {
                uint4 q[sizeof(T) / 2];
                T e[8];
            } u;
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) u.q[i] = reinterpret_cast<const uint4 *>(r)[i];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = as_float<T>(u.e[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = c + i < p.K ? as_float<T>(r[i]) : 0.f;
        }
    }
};
// h of the slots, in rows of ldh floats, a multiple of 8:
struct GatedRows {
    static constexpr int kTop = 14;
    static __device__ __forceinline__ void load(const MoeStream &p, int slot, int c, float (&v)[8]) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (c < p.K) {
            const float4 *r = reinterpret_cast<const float4 *>(p.in + (long long)slot * p.ldh + c);
            a = r[0], b = r[1];
        }
        const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < p.K ? w[i] : 0.f;   // what is behind the row is not h
    }
};
// act(gate) * up of the slices' sums, [ns_in][P][2][ldh]:
struct SlicedRows {
    static constexpr int kTop = 14;
    static __device__ __forceinline__ void load(const MoeStream &p, int slot, int c, float (&v)[8]) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            float a = 0.f, b = 0.f;
            if (c + i < p.K)
                for (int s = 0; s < p.ns_in; ++s) {
                    const float *g = p.in + ((long long)s * p.P + slot) * 2 * p.ldh + c + i;
                    a += g[0], b += g[p.ldh];
                }
            a = act_q8(a, p.act) * b;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i == j) v[j] = a;
        }
    }
};

// The power of two that brings a column's largest magnitude (its bits) to
// [2^to, 2^(to + 1)); at most 2^126, so that the inverse is a normal number.
__device__ __forceinline__ int exponent_for(unsigned top, int to) { return top ? min(126, to + 127 - (int)(top >> 23)) : 0; }
__device__ __forceinline__ float power(int e) { return __uint_as_float((unsigned)(127 + e) << 23); }

__device__ __forceinline__ unsigned largest(const float (&v)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));     // a NaN shows in the products
    return __float_as_uint(m);
}

// Unit u of a column: the eight values whose 16 bytes stand side by side for
// the instructions, and where they do.  Per 64 bytes of codes a column has KC / 8
// pieces of 64 bytes, 16 of them for each of the four threads that share a row.
template <int FMT, class Src>
__device__ __forceinline__ void unit8(const MoeStream &p, int row, int k0, int u, float (&v)[8]) {
    if constexpr (FMT == B200Q_I2) {
        // a word is 16 codes: the values that its instructions 2j, 2j+1 take, j = u & 1
        const int c = k0 + 16 * (u >> 1), j = u & 1;
        float lo[8], hi[8];
        Src::load(p, row, c, lo);
        Src::load(p, row, c + 8, hi);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            v[4 * t] = j ? lo[2 + t] : lo[t];
            v[4 * t + 1] = j ? hi[2 + t] : hi[t];
            v[4 * t + 2] = j ? lo[6 + t] : lo[4 + t];
            v[4 * t + 3] = j ? hi[6 + t] : hi[4 + t];
        }
    } else {
        Src::load(p, row, k0 + 8 * u, v);
    }
}
template <int FMT>
__device__ __forceinline__ int unit_at(int u) {
    if constexpr (FMT == B200Q_I2) return (u >> 5) * 512 + (((u >> 1) & 3) * 2 + (u & 1)) * 64 + ((u >> 3) & 3) * 16;
    constexpr int V = Fmt<FMT>::KC / 8;        // units of a thread's 16 bytes of codes
    return u / (4 * V) * (64 * V) + u % V * 64 + u / V % 4 * 16;
}

// A unit's values, scaled, as 16 bytes of f16 in the order in which fields() takes a
// word of codes apart, and kRest times what is left of them to `rest`: a second
// piece for what the first one rounds off, subnormal first pieces included.
constexpr float kRest = 2048.f;
template <int FMT, int PC>
__device__ __forceinline__ void split(const float (&v)[8], float scale, uint4 &hi, uint4 &rest) {
    constexpr int kOrder[8] = {0, FMT == B200Q_I4 ? 4 : 1, 2, FMT == B200Q_I4 ? 6 : 3,
                               FMT == B200Q_I4 ? 1 : 4, 5, FMT == B200Q_I4 ? 3 : 6, 7};
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = v[kOrder[2 * i]] * scale, b = v[kOrder[2 * i + 1]] * scale;
        const __half2 t = __floats2half2_rn(a, b);
        h[i] = *reinterpret_cast<const uint32_t *>(&t);
        if constexpr (PC == 2) {
            const float2 f = __half22float2(t);
            const __half2 r = __floats2half2_rn((a - f.x) * kRest, (b - f.y) * kRest);
            l[i] = *reinterpret_cast<const uint32_t *>(&r);
        }
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    if constexpr (PC == 2) rest = make_uint4(l[0], l[1], l[2], l[3]);
}

// The sums of rows r and r + 8 of a tile (8 of gate and up, or 16 of down) with
// the column of a slot: written.
__device__ __forceinline__ void put(const MoeStream &p, int slice, int slot, int tile, int r, float a, float b) {
    const long long at = (long long)slice * p.P + slot;
    if (p.down) {
        const int o = tile * 16 + r;
        if (o < p.rows) p.out[at * p.rows + o] = a;
        if (o + 8 < p.rows) p.out[at * p.rows + o + 8] = b;
    } else {
        const int f = tile * 8 + r;
        if (f >= p.rows) return;
        if (p.ns == 1) {
            p.out[at * p.ldh + f] = act_q8(a, p.act) * b;
        } else {
            p.out[at * 2 * p.ldh + f] = a;
            p.out[(at * 2 + 1) * p.ldh + f] = b;
        }
    }
}

// The products of a thread's 16 bytes of codes (of MT tiles, rows g and g + 8)
// with N x 8 columns of the NT x 8 that have sums; `from(nt)` is where this
// thread's column of tile nt has its values, its second pieces `plane` bytes
// further.  The words take NA accumulators in turn: an instruction waits for the
// one before it on the same accumulator.  Two pieces: the first ones' sums are
// taken out of the accumulator after every word of codes, the second ones are in
// `rest`, kRest times.
template <int FMT, int N, int NT, int MT, int PC, int NA, class From>
__device__ __forceinline__ void chunk_products(const uint4 (&q)[MT][2], From from, int plane, float (&sum)[MT][NT][4],
                                               float (&accs)[NA][MT][NT][4],
                                               float (&rests)[PC == 2 ? NA : 1][PC == 2 ? MT : 1][PC == 2 ? NT : 1][4]) {
    constexpr int MMAS = Fmt<FMT>::MMAS;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        float (&acc)[MT][NT][4] = accs[w % NA];
        auto &rest = rests[PC == 2 ? w % NA : 0];
        uint32_t a[MT][MMAS][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint4 &c0 = q[m][0], &c1 = q[m][1];
            const uint32_t w0 = w == 0 ? c0.x : w == 1 ? c0.y : w == 2 ? c0.z : c0.w;
            const uint32_t w1 = w == 0 ? c1.x : w == 1 ? c1.y : w == 2 ? c1.z : c1.w;
#pragma unroll
            for (int t = 0; t < MMAS; ++t) {
                fields<FMT>(w0, t, a[m][t][0], a[m][t][2]);
                fields<FMT>(w1, t, a[m][t][1], a[m][t][3]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < N; ++nt) {
#pragma unroll
            for (int pc = 0; pc < PC; ++pc) {
                const uint8_t *at = from(nt) + pc * plane;
                auto to = [&](int m) -> float (&)[4] { return pc ? rest[PC == 2 ? m : 0][PC == 2 ? nt : 0] : acc[m][nt]; };
                if constexpr (MMAS == 1) {
                    const uint2 b = *reinterpret_cast<const uint2 *>(at + (w >> 1) * 64 + (w & 1) * 8);
#pragma unroll
                    for (int m = 0; m < MT; ++m) mma_f16(to(m), a[m][0][0], a[m][0][1], a[m][0][2], a[m][0][3], b.x, b.y);
                } else {
#pragma unroll
                    for (int t = 0; t < MMAS; t += 2) {
                        const uint4 b = *reinterpret_cast<const uint4 *>(at + (w * (MMAS / 2) + t / 2) * 64);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            mma_f16(to(m), a[m][t][0], a[m][t][1], a[m][t][2], a[m][t][3], b.x, b.y);
                            mma_f16(to(m), a[m][t + 1][0], a[m][t + 1][1], a[m][t + 1][2], a[m][t + 1][3], b.z, b.w);
                        }
                    }
                }
            }
            if constexpr (PC == 2) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[m][nt][i] += acc[m][nt][i], acc[m][nt][i] = 0.f;
            }
        }
    }
}

// ---------------------------------------------------------------- few columns
// Up to 8 columns of an expert, those of a few chunks at a time in shared memory.
constexpr int kFewColumns = kMoeFewColumns, kFewHeld = 16;  // of a chunk; of the chunks that are staged together

struct FewColumns {
    unsigned top[kFewHeld];                    // the largest magnitude
    float unscale[kFewHeld];                   // the inverse scale
    const float *scales[kFewHeld][2];          // of a chunk: its rows' scales, gate and up, or down twice
};

// W: warps of a block; AHEAD: lines in a warp's ring.
template <int W, int AHEAD> struct FewShape {
    static constexpr int kRing = W * AHEAD * 2048;
    static constexpr int kBarsAt = kRing;
    static constexpr int kRedAt = kBarsAt + W * AHEAD * 8 + 16;        // and the columns' barrier
    static constexpr int kRedTile = kFewColumns * kRedPitch;           // floats of a warp's tile
    static constexpr int kRed = 2 * W * kRedTile * 4;                  // two sets, used in turn; the plan's scratch before
    static constexpr int kColumnsAt = kRedAt + kRed;
    static constexpr int kPlanAt = kColumnsAt + (int)sizeof(FewColumns);
    static constexpr int kB = (kPlanAt + (int)sizeof(Plan) + 127) / 128 * 128;
    static_assert(sizeof(PlanScratch) <= kRed, "the plan's scratch lies where the sums will");
};

__device__ __forceinline__ unsigned long long global_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Whether the barrier's phase ended within the limit.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, unsigned long long limit_ns) {
    unsigned long long t0 = 0;
#pragma unroll 1
    for (uint32_t it = 0;; ++it) {
        uint32_t done;
        asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                     : "=r"(done)
                     : "r"(bar), "r"(parity)
                     : "memory");
        if (done) return true;
        if (it == 0) t0 = global_ns();
        if ((it & 255) == 255 && global_ns() - t0 > limit_ns) return false;
    }
}

constexpr unsigned long long kMoeDrainNs = 250000000ull;               // for copies in flight, after giving up

// The tensor maps lie in memory that a copy wrote (cudaMemcpyAsync, when the handle
// was made), not in a kernel's parameters: a block acquires those of its chunks, c0 to
// c1, before its first copy, or a map that lay at an address before, of a freed layer, may
// serve.  Once for the block, before a barrier of its own: every warp for itself takes the
// same maps again and again (one token through 8 int4 experts of 6144 / 2048: 46.2 us so, 43.3 us by block).
__device__ __forceinline__ void acquire_maps(const MoeStream &p, const Plan &pl, int c0, int c1, bool wide) {
    const int n = p.down ? 1 : 2;
    for (int i = threadIdx.x; i < n * (c1 - c0 + 1); i += blockDim.x) {
        const Expert &e = p.table[pl.expert[c0 + (n == 2 ? i >> 1 : i)]];
        const CUtensorMap *map = (wide ? e.wide : e.map) + (n == 2 ? i & 1 : 2);
        asm volatile("fence.proxy.tensormap::generic.acquire.sys [%0], 128;" ::"l"(map) : "memory");
    }
}

// A box of 8 rows x 128 bytes of codes to shared memory, swizzled.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3}], [%4], "
        "%5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void copy_bulk(uint32_t dst, const void *src, int bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
                 "r"(bar)
                 : "memory");
}

// n rows, lines l0 .. l1-1 of them, into shared memory as columns; row_of(c) is
// column c's.  First their largest magnitudes, then once more to scale them.
// Called by the whole block; ends with a barrier.
template <int FMT, int PC, class Src, class RowOf>
__device__ __forceinline__ void stage_from(const MoeStream &p, RowOf row_of, int n, int l0, int l1, uint8_t *B, FewColumns &cl) {
    constexpr int KC = Fmt<FMT>::KC;
    const int units = (l1 - l0) * KC;          // of a column: KC to a line
    const int k0 = l0 * 8 * KC, tid = threadIdx.x, lane = tid & 31;
    int lg = 5;                                // 2^lg threads take a column
    while (1 << lg < units && 1 << lg < (int)blockDim.x) ++lg;
    const int sub = tid & ((1 << lg) - 1), c0 = tid >> lg, step = (int)blockDim.x >> lg;
    if (tid < kFewHeld) cl.top[tid] = 0u;
    __syncthreads();
#pragma unroll 1
    for (int c = c0; c < n; c += step) {
        const int row = row_of(c);
        unsigned m = 0;
#pragma unroll 1
        for (int u = sub; u < units; u += 1 << lg) {
            float v[8];
            Src::load(p, row, k0 + 8 * u, v);
            m = max(m, largest(v));
        }
        m = __reduce_max_sync(kAll, m);
        if (lane == 0) atomicMax(&cl.top[c], m);
    }
    __syncthreads();
#pragma unroll 1
    for (int c = c0; c < n; c += step) {
        const int row = row_of(c), up = exponent_for(cl.top[c], Src::kTop);
        const float scale = power(up);
        uint8_t *to = B + c * p.pitch;
#pragma unroll 1
        for (int u = sub; u < units; u += 1 << lg) {
            float v[8];
            uint4 hi, rest;
            unit8<FMT, Src>(p, row, k0, u, v);
            split<FMT, PC>(v, scale, hi, rest);
            *reinterpret_cast<uint4 *>(to + unit_at<FMT>(u)) = hi;
            if constexpr (PC == 2) *reinterpret_cast<uint4 *>(to + unit_at<FMT>(u) + p.held * p.pitch) = rest;
        }
        if (sub == 0) cl.unscale[c] = power(-up);
    }
    __syncthreads();
}

template <int FMT, int PC, class RowOf>
__device__ __forceinline__ void stage(const MoeStream &p, RowOf row_of, int n, int l0, int l1, uint8_t *B, FewColumns &cl) {
    if (p.down) {
        if (p.ns_in == 1) stage_from<FMT, PC, GatedRows>(p, row_of, n, l0, l1, B, cl);
        else stage_from<FMT, PC, SlicedRows>(p, row_of, n, l0, l1, B, cl);
    } else if constexpr (PC == 2) {            // with two pieces 16-bit rows are only h
        stage_from<FMT, PC, TokenRows<float>>(p, row_of, n, l0, l1, B, cl);
    } else {
        if (p.type == B200Q_T_F16) stage_from<FMT, PC, TokenRows<__half>>(p, row_of, n, l0, l1, B, cl);
        else stage_from<FMT, PC, TokenRows<__nv_bfloat16>>(p, row_of, n, l0, l1, B, cl);
    }
}

template <int FMT, int PC, int W, int AHEAD>
__global__ void __launch_bounds__(32 * W, 16 / W) moe_few_kernel(const __grid_constant__ MoeStream p) {
    using Sh = FewShape<W, AHEAD>;
    constexpr int KC = Fmt<FMT>::KC;
    extern __shared__ __align__(1024) uint8_t smem[];
    float *red = reinterpret_cast<float *>(smem + Sh::kRedAt);
    FewColumns &cl = *reinterpret_cast<FewColumns *>(smem + Sh::kColumnsAt);
    Plan &pl = *reinterpret_cast<Plan *>(smem + Sh::kPlanAt);
    uint8_t *B = smem + Sh::kB;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (AHEAD * 2048);
    const uint32_t bars = (uint32_t)__cvta_generic_to_shared(smem + Sh::kBarsAt) + warp * (AHEAD * 8);
    // The lanes' rows of a box are not in order: two rows that a quarter of a warp
    // reads together have their 16 bytes in different banks.
    const int row = (g & 1) << 2 | g >> 1;

    // Addresses that the kernel will wait for one after the other, asked for
    // together: their pages have to be found.
    if (tid == 0) prefetch(p.ids);
    if (tid == 32) prefetch(p.table);
    if (tid == 64) prefetch(p.down ? (const void *)p.in : p.x);
    if (tid == 96) prefetch(p.out);
    const uint32_t colbar = (uint32_t)__cvta_generic_to_shared(smem + Sh::kBarsAt + W * AHEAD * 8);
    if (lane == 0) {                           // the warp's own barriers
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bars + 8 * i) : "memory");
        if (warp == 0) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(colbar) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    // The ids may come from the kernel before the call's first; the others follow
    // it, and the ids were there when it began.
    const bool first_kernel = !p.down && !p.prepared;
    if (first_kernel) dependency_wait();
    make_plan(p, pl, *reinterpret_cast<PlanScratch *>(red));
    // the tokens' rows are the columns where all of them have room
    const bool tokens = !p.down && p.ns == 1 && p.S <= p.held;
    // an even run of the tiles; their number is below 2^31
    const int all = pl.chunks * p.ns * p.tiles, each = p.by_grid(all), more = all - each * (int)gridDim.x;
    const int lo = (int)blockIdx.x * each + min((int)blockIdx.x, more), hi = lo + each + ((int)blockIdx.x < more ? 1 : 0);
    if (lo < hi) acquire_maps(p, pl, p.by_tiles(lo) / p.ns, p.by_tiles(hi - 1) / p.ns, false);
    __syncthreads();
    const int wk = 1 << p.wk, kw = warp & (wk - 1), groups = W >> p.wk, wm = warp >> p.wk;
    auto first_line = [&](int slice) { return p.ns == 1 ? (slice ? p.lines : 0) : (int)((long long)slice * p.lines / p.ns); };

    // the copy cursor: this warp's next line
    int fu = lo + wm, fline = 0, fl1 = 0, fy = 0, fslot = 0;
    const CUtensorMap *map = nullptr;          // of gate or down; the one of up is the next
    const uint64_t policy = stream_policy();
    auto open = [&]() {                        // the cursor's tile, or a later one that has a line for this warp
#pragma unroll 1
        for (; fu < hi; fu += groups) {
            const int cs = p.by_tiles(fu), c = p.ns == 1 ? cs : cs / p.ns, sl = cs - c * p.ns;
            fline = first_line(sl) + kw;
            fl1 = first_line(sl + 1);
            if (fline >= fl1) continue;
            map = p.table[pl.expert[c]].map + (p.down ? 2 : 0);
            fy = (fu - cs * p.tiles) * (p.down ? 16 : 8);
            return;
        }
    };
    auto copy_line = [&]() {
        if (fu < hi) {
            if (lane == 0) {
                const uint32_t to = ring + fslot * 2048, bar = bars + 8 * fslot;
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], 2048;" ::"r"(bar) : "memory");
                copy_box(to, map, fline * 128, fy, bar, policy);
                copy_box(to + 1024, p.down ? map : map + 1, fline * 128, p.down ? fy + 8 : fy, bar, policy);
            }
            if (++fslot == AHEAD) fslot = 0;
            if ((fline += wk) >= fl1) {
                fu += groups;
                open();
            }
        }
    };
    open();
#pragma unroll 1
    for (int i = 0; i < AHEAD; ++i) copy_line();
    if (!first_kernel) dependency_wait();
    let_dependents_start();

    const uint8_t *mine = smem + warp * (AHEAD * 2048) + row * 128 + ((tig ^ row) << 4);
    int slot = 0, set = 0, u = lo + wm;        // the warp's tiles follow each other as the cursor's do
    uint32_t parity = 0, colparity = 0;
    bool ok = true;                            // false: a copy did not come, the rest is not waited for
#pragma unroll 1
    for (int u0 = lo; u0 < hi;) {              // the block's tiles whose columns are staged together
        const int cs0 = p.by_tiles(u0), c0 = p.ns == 1 ? cs0 : cs0 / p.ns, slice = cs0 - c0 * p.ns;
        const int l0 = first_line(slice), l1 = first_line(slice + 1);
        const unsigned short *order = pl.order + pl.first[c0];
        int held = pl.n[c0], chunks = 1, u1 = (cs0 + 1) * p.tiles;
        if (p.ns == 1) {
#pragma unroll 1
            for (; u1 < hi && chunks < kFewHeld && (tokens || held + pl.n[c0 + chunks] <= p.held); u1 += p.tiles)
                held += pl.n[c0 + chunks], ++chunks;
        }
        u1 = min(u1, hi);
        __syncthreads();                       // the columns before are read, and the plan's scratch
        if (tid < chunks) {
            const Expert &e = p.table[pl.expert[c0 + tid]];
            cl.scales[tid][0] = e.scales[p.down ? 2 : 0];
            cl.scales[tid][1] = p.down ? e.scales[2] + 8 : e.scales[1];
        }
        auto row_of = [&](int c) { return tokens ? c : p.down ? order[c] : p.by_k(order[c]); };
        const int columns = tokens ? p.S : held;
        if (tokens && u0 != lo) {
            __syncthreads();
        } else if (p.prepared) {
            const int bytes = (l1 - l0) * (16 * KC);
            if (tid == 0 && ok) {
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(colbar), "r"(columns * PC * bytes + p.withheld) : "memory");
#pragma unroll 1
                for (int c = 0; c < columns * PC; ++c) {               // first pieces, then second ones
                    const int col = c < columns ? c : c - columns;
                    const uint8_t *from = p.cols + ((long long)(row_of(col) * PC + (c < columns ? 0 : 1)) * p.lines + l0) * (16 * KC);
                    copy_bulk((uint32_t)__cvta_generic_to_shared(B) + (col + (c < columns ? 0 : p.held)) * p.pitch, from, bytes, colbar);
                }
            }
            if (tid < columns) cl.unscale[tid] = p.info[row_of(tid)];
            if (ok) ok = mbar_wait(colbar, colparity, p.wait_ns);
            colparity ^= 1;
            __syncthreads();
        } else {
            stage<FMT, PC>(p, row_of, columns, l0, l1, B, cl);
        }
#pragma unroll 1
        for (; u < u1; u += groups) {
            const int cs = p.by_tiles(u), at = p.ns == 1 ? cs - c0 : 0, tile = u - cs * p.tiles;
            const int n = pl.n[c0 + at], first = pl.first[c0 + at] - pl.first[c0];
            auto column = [&](int c) { return tokens ? p.by_k(order[first + c]) : first + c; };
            // the scales of rows r and r + 8, fetched now, used at the end; rows past the last have scale 0
            const int r = wk == 1 ? row : tid & 7, o = tile * (p.down ? 16 : 8) + r;
            const float sa = cl.scales[at][0][o], sb = cl.scales[at][1][o];
            float sum[1][1][4] = {};
            // a column past the chunk's is computed and not stored
            const uint8_t *xb = B + column(min(g, n - 1)) * p.pitch + tig * 16 + kw * (16 * KC);
#pragma unroll 1
            for (int line = l0 + kw; line < l1; line += wk, xb += wk * (16 * KC)) {
                if (ok) ok = mbar_wait(bars + 8 * slot, parity, p.wait_ns);
                const uint8_t *from = mine + slot * 2048, *from2 = reinterpret_cast<const uint8_t *>((uintptr_t)from ^ 64);
                uint4 q[1][2], next[1][2];     // [tile][row half]
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    q[0][i] = *reinterpret_cast<const uint4 *>(from + i * 1024);
                    next[0][i] = *reinterpret_cast<const uint4 *>(from2 + i * 1024);
                }
                __syncwarp();                  // the slot is read
                if (ok) {                      // otherwise what is in flight stays as it is told below
                    if (++slot == AHEAD) slot = 0, parity ^= 1;
                    copy_line();
                }
                constexpr int NA = PC == 2 ? 2 : 4;
                float acc[NA][1][1][4] = {}, rest[PC == 2 ? NA : 1][1][1][4] = {};
                chunk_products<FMT, 1, 1, 1, PC, NA>(q, [&](int) { return xb; }, p.held * p.pitch, sum, acc, rest);
                chunk_products<FMT, 1, 1, 1, PC, NA>(next, [&](int) { return xb + 8 * KC; }, p.held * p.pitch, sum, acc, rest);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (PC == 2) sum[0][0][i] = fmaf(rest[0][0][0][i] + rest[1][0][0][i], 1.f / kRest, sum[0][0][i]);
                    else sum[0][0][i] += (acc[0][0][0][i] + acc[1][0][0][i]) + (acc[2][0][0][i] + acc[3][0][0][i]);
                }
            }
            float a0 = sum[0][0][0], b0 = sum[0][0][2], a1 = sum[0][0][1], b1 = sum[0][0][3];
            int col = 2 * tig, stride = 1, end = min(n, col + 2);      // the columns that this thread writes, row r of the tile
            const float *part = red + (set * W + wm * wk) * Sh::kRedTile + r;
            if (wk > 1) {
                // [column][row] of this warp's part, added over the tile's warps in order; the two sets
                // take turns, so that one barrier per tile is enough
                float *to = red + (set * W + warp) * Sh::kRedTile + 2 * tig * kRedPitch + row;
                to[0] = a0, to[kRedPitch] = a1, to[8] = b0, to[kRedPitch + 8] = b1;
                asm volatile("bar.sync %0, %1;" ::"r"(1 + wm), "r"(wk * 32) : "memory");
                col = (kw * 32 + lane) >> 3, stride = wk * 4, end = n;
                set ^= 1;
            }
#pragma unroll 1
            for (; col < end; col += stride) {
                if (wk > 1) {
                    a0 = b0 = 0.f;
                    for (int w = 0; w < wk; ++w) a0 += part[col * kRedPitch + w * Sh::kRedTile], b0 += part[col * kRedPitch + w * Sh::kRedTile + 8];
                }
                const int b = column(col);
                const float un = cl.unscale[b];
                put(p, slice, order[first + col], tile, r, a0 * sa * un, b0 * sb * un);
                a0 = a1, b0 = b1;
            }
        }
        u0 = u1;
    }
    if (!ok) {
        // gave up: say so, and let the copies in flight land
        if (lane == 0) atomicCAS(p.err, 0u, (unsigned)(-B200Q_ETIMEOUT));
#pragma unroll 1
        for (int i = 0; i < AHEAD; ++i) mbar_wait(bars + 8 * i, i < slot ? parity ^ 1 : parity, kMoeDrainNs);
        if (p.prepared) mbar_wait(colbar, colparity ^ 1, kMoeDrainNs);
    }
}

// ---------------------------------------------------------------- many columns
// Up to 32 columns of an expert, prepared in memory once and copied line by line
// beside the codes, in stages that the whole block shares: a warp keeps the sums
// of 16 rows with all columns over the rows' whole length.
template <int N> struct Count {
    static constexpr int value = N;
};
constexpr int kManyWarps = 16, kManyThreads = 32 * kManyWarps, kManyHeld = 8;
template <int FMT, int PC> constexpr int kManyColumns = FMT == B200Q_I2 && PC == 2 ? 16 : 32;
template <int FMT, int PC> constexpr int kManyStages = FMT == B200Q_I8 || (FMT == B200Q_I4 && PC == 1) ? 4 : 3;
template <int FMT, int PC> struct ManyShape {
    static constexpr int kPitch = 16 * Fmt<FMT>::KC + 64;              // of a column's line: no bank conflicts
    static constexpr int kPlane = kManyColumns<FMT, PC> * kPitch;
    static constexpr int kCodes = kManyWarps * 2048;
    static constexpr int kStage = kCodes + PC * kPlane;
    static_assert(kStage % 1024 == 0, "a box of codes is swizzled by its address");
    static constexpr int kBarsAt = kManyStages<FMT, PC> * kStage;      // the plan's scratch lies in the stages before
    static constexpr int kPlanAt = kBarsAt + 2 * 8 * kManyStages<FMT, PC>;
    static constexpr int kBytes = kPlanAt + (int)sizeof(Plan);
};

// A row of the tokens, or of h, per block, as pieces in the order of the
// instructions; its inverse scale to info.  Few columns read rows: [row]
// [piece][line][16 KC].  ORDERED, for many: where the plan has the row's slots, a
// line of all of them side by side, [piece][line][place][kPitch], so that one copy
// brings a chunk's.
template <int FMT, int PC, bool ORDERED, class Src>
__global__ void __launch_bounds__(256) moe_prepare_kernel(const __grid_constant__ MoeStream p, uint8_t *cols, float *info) {
    constexpr int KC = Fmt<FMT>::KC, kPitch = ManyShape<FMT, PC>::kPitch;
    __shared__ unsigned tops[8];
    __shared__ int places[kMoeMaxK];
    dependency_wait();
    let_dependents_start();
    const int row = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, units = p.lines * KC;
    const int slots = ORDERED && !p.down ? p.k : 1;                     // of this row
    if (p.down) {
        const int e = p.ids[row];
        if (e < 0 || e >= p.E) return;         // an empty slot has no h
    }
    if constexpr (ORDERED) {
        // a slot's place: the slots of lower experts, and of its own before it
#pragma unroll 1
        for (int j = warp; j < slots; j += 8) {
            const int slot = row * slots + j, e = p.ids[slot];
            int place = 0;
#pragma unroll 1
            for (int i = lane; i < p.P; i += 32) {
                const int o = p.ids[i];
                place += o >= 0 && o < p.E && (o < e || (o == e && i < slot)) ? 1 : 0;
            }
            place = __reduce_add_sync(kAll, place);
            if (lane == 0) places[j] = e >= 0 && e < p.E ? place : -1;
        }
    }
    unsigned m = 0;
#pragma unroll 1
    for (int u0 = threadIdx.x; u0 < units; u0 += 3 * 256) {
        float v[3][8];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
            if (u0 + i * 256 < units) Src::load(p, row, 8 * (u0 + i * 256), v[i]);
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) m = max(m, largest(v[i]));
    }
    m = __reduce_max_sync(kAll, m);
    if (lane == 0) tops[warp] = m;
    __syncthreads();
    m = __reduce_max_sync(kAll, tops[lane & 7]);
    const int up = exponent_for(m, Src::kTop);
    const float scale = power(up);
#pragma unroll 1
    for (int u = threadIdx.x; u < units; u += 256) {
        float v[8];
        uint4 hi, rest;
        unit8<FMT, Src>(p, row, 0, u, v);
        split<FMT, PC>(v, scale, hi, rest);
        if constexpr (ORDERED) {
            const int line = unit_at<FMT>(u) / (16 * KC), in = unit_at<FMT>(u) - line * (16 * KC);
#pragma unroll 1
            for (int j = 0; j < slots; ++j) {
                if (places[j] < 0) continue;
                uint8_t *to = cols + ((long long)line * p.P + places[j]) * kPitch + in;
                *reinterpret_cast<uint4 *>(to) = hi;
                if constexpr (PC == 2) *reinterpret_cast<uint4 *>(to + (long long)p.lines * p.P * kPitch) = rest;
            }
        } else {
            uint8_t *to = cols + (long long)row * PC * p.lines * (16 * KC) + unit_at<FMT>(u);
            *reinterpret_cast<uint4 *>(to) = hi;
            if constexpr (PC == 2) *reinterpret_cast<uint4 *>(to + (long long)p.lines * (16 * KC)) = rest;
        }
    }
    if (threadIdx.x < slots) {
        const int at = ORDERED ? places[threadIdx.x] : row;
        if (at >= 0) info[at] = power(-up);
    }
}

template <int FMT, int PC>
__global__ void __launch_bounds__(kManyThreads, 1) moe_many_kernel(const __grid_constant__ MoeStream p) {
    using Sh = ManyShape<FMT, PC>;
    constexpr int KC = Fmt<FMT>::KC, NT = kManyColumns<FMT, PC> / 8, STAGES = kManyStages<FMT, PC>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Plan &pl = *reinterpret_cast<Plan *>(smem + Sh::kPlanAt);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
    const int row = (g & 1) << 2 | g >> 1;     // of a box: as in the kernel for few columns
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem), full = base + Sh::kBarsAt, empty = full + 8 * STAGES;

    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < 2 * STAGES; ++i)   // five warps bring a stage, all let go of it
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(full + 8 * i), "r"(i < STAGES ? 5 : kManyWarps) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // the ids were there when the kernel that prepares the rows began
    make_plan(p, pl, *reinterpret_cast<PlanScratch *>(smem));
    // A round: up to 16 tiles of one chunk, a warp each, over the whole length of the
    // rows; a block takes an even run of rounds.  (More and shorter rounds, so that no
    // block has one more than others: no gain, since the boxes then bring rows twice.)
    const int rounds = (p.tiles + kManyWarps - 1) / kManyWarps;        // of a chunk
    const int all = pl.chunks * rounds, each = p.by_grid(all), more = all - each * (int)gridDim.x;
    const int lo = (int)blockIdx.x * each + min((int)blockIdx.x, more), hi = lo + each + ((int)blockIdx.x < more ? 1 : 0);
    if (lo < hi) acquire_maps(p, pl, p.by_rounds(lo), p.by_rounds(hi - 1), true);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");       // the scratch was written here, the stages are by copies
    __syncthreads();
    dependency_wait();
    let_dependents_start();
    auto tiles_of = [&](int u, int &c, int &from) {                    // round u's chunk, first tile and tiles
        c = p.by_rounds(u);
        from = (u - c * rounds) * kManyWarps;
        return min(p.tiles - from, kManyWarps);
    };

    // A stage's copies: the codes in four boxes of 64 rows (8 tiles of gate or of up,
    // or 4 of down; a round's last box may bring rows that it does not want), one by
    // each of the first four warps, and the columns by the fifth.
    int fu = lo, fline = 0, fstage = 0, fbytes = 0, fy = 0;
    const CUtensorMap *map = nullptr;
    const uint8_t *from = nullptr;
    const uint64_t policy = stream_policy();
    const long long line_bytes = (long long)p.P * Sh::kPitch;
    auto open = [&]() {
        if (fu >= hi) return;
        int c, first;
        const int tiles = tiles_of(fu, c, first);
        fline = 0;
        if (warp < 4) {
            const int box = p.down ? 4 : 8, at = p.down ? warp : warp & 1;          // tiles of a box, this one
            map = p.table[pl.expert[c]].wide + (p.down ? 2 : warp >> 1);
            fy = (first + at * box) * (p.down ? 16 : 8);
            fbytes = at * box < tiles ? 8192 : 0;
        } else {
            from = p.cols + pl.first[c] * Sh::kPitch;
            fbytes = pl.n[c] * Sh::kPitch;
        }
    };
    auto copy_stage = [&]() {                  // lane 0 of the first five warps
        if (fu >= hi) return;
        const uint32_t to = base + fstage * Sh::kStage, bar = full + 8 * fstage;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(warp < 4 ? fbytes : PC * fbytes + p.withheld) : "memory");
        if (warp < 4) {
            if (fbytes) copy_box(to + warp * 8192, map, fline * 128, fy, bar, policy);
        } else {
#pragma unroll
            for (int pc = 0; pc < PC; ++pc)
                copy_bulk(to + Sh::kCodes + pc * Sh::kPlane, from + (pc * p.lines + fline) * line_bytes, fbytes, bar);
        }
        if (++fstage == STAGES) fstage = 0;
        if (++fline == p.lines) {
            ++fu;
            open();
        }
    };
    if (warp < 5 && lane == 0) {
        open();
#pragma unroll 1
        for (int i = 0; i < STAGES; ++i) copy_stage();
    }
    int stage = 0, before = 0;                 // the stage that is read, the one that was
    uint32_t parity = 0, parity_before = 0;
    bool ok = true;                            // false: a copy did not come, or a warp did not let go: nothing more is waited for
#pragma unroll 1
    for (int u = lo; u < hi; ++u) {
        int chunk, first;
        const bool mine = warp < tiles_of(u, chunk, first);
        const int n = pl.n[chunk], tile = first + warp;
        // One piece: the sums are taken out of the accumulators after every kManyHeld lines.  An instruction drops up to
        // an accumulator's last place, so that what is lost of a sum grows with the instructions between (64 of int4: 4e-6
        // of their sum |deq x|); over the whole row it would grow with the row.  Two: after every word of codes.
        constexpr int NA = PC == 2 ? 1 : 2;
        float sum[1][NT][4] = {}, acc[NA][1][NT][4] = {}, sa = 0.f, sb = 0.f;
        if (mine) {
            const Expert &e = p.table[pl.expert[chunk]];
            const int o = tile * (p.down ? 16 : 8) + row;
            sa = (p.down ? e.scales[2] : e.scales[0])[o];
            sb = (p.down ? e.scales[2] + 8 : e.scales[1])[o];
        }
#pragma unroll 1
        for (int line = 0; line < p.lines; ++line) {
            if (ok) ok = mbar_wait(full + 8 * stage, parity, p.wait_ns);
            const uint8_t *at = smem + stage * Sh::kStage;
            // N: the tiles of columns that the chunk has; without a branch between their instructions
            auto products = [&](auto tiles) {
                constexpr int N = decltype(tiles)::value;
                float rest[1][1][PC == 2 ? NT : 1][4] = {};
                // rows 8-15 of a tile lie behind rows 0-7, or are up's, in the third and fourth box
                const uint8_t *codes = at + warp * (p.down ? 2048 : 1024) + row * 128 + ((tig ^ row) << 4);
                const int second = p.down ? 1024 : 16384;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint8_t *from = reinterpret_cast<const uint8_t *>((uintptr_t)codes ^ (half * 64));
                    uint4 q[1][2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) q[0][i] = *reinterpret_cast<const uint4 *>(from + i * second);
                    const uint8_t *b = at + Sh::kCodes + g * Sh::kPitch + half * (8 * KC) + tig * 16;
                    chunk_products<FMT, N, NT, 1, PC, NA>(q, [&](int nt) { return b + nt * (8 * Sh::kPitch); }, Sh::kPlane, sum, acc, rest);
                }
                if constexpr (PC == 2) {
#pragma unroll
                    for (int nt = 0; nt < N; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum[0][nt][i] = fmaf(rest[0][0][nt][i], 1.f / kRest, sum[0][nt][i]);
                }
            };
            if (mine) {
                if (n <= 8) products(Count<1>{});
                else if (n <= 16) products(Count<2>{});
                else if (NT > 2 && n <= 24) products(Count<NT < 3 ? NT : 3>{});
                else products(Count<NT>{});
            }
            __syncwarp();
            if (lane == 0 && ok) {
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(empty + 8 * stage) : "memory");
                // the stage before this one is let go by all, or soon: filled again
                if (warp < 5 && (u != lo || line)) {
                    if (fu < hi) ok = mbar_wait(empty + 8 * before, parity_before, p.wait_ns);
                    if (ok) copy_stage();
                }
            }
            if (ok) {                          // otherwise what is in flight stays as it is told below
                before = stage, parity_before = parity;
                if (++stage == STAGES) stage = 0, parity ^= 1;
            }
            if constexpr (PC == 1) {
                if ((line + 1) % kManyHeld == 0 || line + 1 == p.lines) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            sum[0][nt][i] += acc[0][0][nt][i] + acc[1][0][nt][i];
                            acc[0][0][nt][i] = acc[1][0][nt][i] = 0.f;
                        }
                }
            }
        }
        if (mine) {
            const unsigned short *order = pl.order + pl.first[chunk];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = nt * 8 + 2 * tig + j;
                    if (c < n) {
                        const float un = p.info[pl.first[chunk] + c];
                        put(p, 0, order[c], tile, row, sum[0][nt][j] * sa * un, sum[0][nt][2 + j] * sb * un);
                    }
                }
        }
    }
    if (!ok) {
        // gave up: say so, and let the copies in flight land
        if (lane == 0) atomicCAS(p.err, 0u, (unsigned)(-B200Q_ETIMEOUT));
#pragma unroll 1
        for (int i = 0; i < STAGES; ++i) mbar_wait(full + 8 * i, i < stage ? parity ^ 1 : parity, kMoeDrainNs);
    }
}

}  // namespace

// ---------------------------------------------------------------- launches
template <int FMT, int PC>
cudaError_t moe_start(const MoeStream &p, const MoeWay &w, int n_sms, cudaStream_t st) {
    auto go = [&](auto kernel) {
        cudaError_t e = allow_dynamic_smem((const void *)kernel, 227 * 1024);
        return e != cudaSuccess ? e : launch_dependent(kernel, dim3(n_sms * w.blocks), 32 * w.warps, w.smem, st, p);
    };
    if (w.kind == 2) return go(moe_many_kernel<FMT, PC>);
    if (w.kind == 1) return go(moe_few_kernel<FMT, PC, 8, 4>);
    return go(moe_few_kernel<FMT, PC, 16, 3>);
}

template <int FMT>
cudaError_t moe_launch_stream(const MoeStream &p, const MoeWay &w, int n_sms, cudaStream_t st) {
    return moe_pieces(p.type, p.down) == 2 ? moe_start<FMT, 2>(p, w, n_sms, st) : moe_start<FMT, 1>(p, w, n_sms, st);
}

template <int FMT>
cudaError_t moe_launch_prepare(const MoeStream &p, int rows, bool ordered, uint8_t *cols, float *info, cudaStream_t st) {
    auto go = [&](auto kernel) { return launch_dependent(kernel, dim3(rows), 256, 0, st, p, cols, info); };
    if (!ordered) {                            // few columns: the tokens' rows
        if (p.type == B200Q_T_F32) return go(moe_prepare_kernel<FMT, 2, false, TokenRows<float>>);
        if (p.type == B200Q_T_F16) return go(moe_prepare_kernel<FMT, 1, false, TokenRows<__half>>);
        return go(moe_prepare_kernel<FMT, 1, false, TokenRows<__nv_bfloat16>>);
    }
    if (p.down) return moe_pieces(p.type, true) == 2 ? go(moe_prepare_kernel<FMT, 2, true, GatedRows>) : go(moe_prepare_kernel<FMT, 1, true, GatedRows>);
    if (p.type == B200Q_T_F32) return go(moe_prepare_kernel<FMT, 2, true, TokenRows<float>>);
    if (p.type == B200Q_T_F16) return go(moe_prepare_kernel<FMT, 1, true, TokenRows<__half>>);
    return go(moe_prepare_kernel<FMT, 1, true, TokenRows<__nv_bfloat16>>);
}

// kind 0 and 1: as many columns as there are tokens, at most 8, and slices that
// keep them within what the ring leaves of the shared memory.
template <int FMT>
MoeWay moe_way_of(int kind, int pieces, int S, int lines) {
    constexpr int KC = Fmt<FMT>::KC;
    MoeWay w{};
    w.kind = kind;
    w.ns = 1;
    w.warps = kind == 1 ? 8 : 16;
    w.blocks = kind == 1 ? 2 : 1;
    if (kind == 2) {
        w.nc = pieces == 2 ? kManyColumns<FMT, 2> : kManyColumns<FMT, 1>;
        w.smem = pieces == 2 ? ManyShape<FMT, 2>::kBytes : ManyShape<FMT, 1>::kBytes;
        static_assert(ManyShape<FMT, 2>::kBytes <= 227 * 1024 && ManyShape<FMT, 1>::kBytes <= 227 * 1024, "shared memory");
        return w;
    }
    w.nc = S < kFewColumns ? S : kFewColumns;
    const size_t fixed = kind ? FewShape<8, 4>::kB : FewShape<16, 3>::kB, room = (kind ? 113 * 1024 : 227 * 1024) - fixed;
    // a column is 64 bytes off a 128-byte multiple: no bank conflicts
    auto most = [&](int ns) {
        const long long n = (long long)room / (((lines + ns - 1ll) / ns * 16 * KC + 64) * pieces);
        return (int)(n < kFewHeld ? n : kFewHeld);
    };
    while (most(w.ns) < w.nc) ++w.ns;
    w.held = most(w.ns);
    w.pitch = (lines + w.ns - 1) / w.ns * 16 * KC + 64;
    w.smem = fixed + (size_t)w.pitch * w.held * pieces;
    return w;
}

}  // namespace qwq
