// The experts' layer for a few tokens, routed on the device.
//     h[s,j] = act(gate_e x[s]) * (up_e x[s]),   y[s] = res[s] + sum_j wts[s,j] down_e h[s,j],   e = ids[s,j]
//
// Bound: HBM, the three matrices of every expert that some token has, each read
// once.  A slot (s, j) is a column of its expert's products.  Three launches: gate
// and up, down, and the weighted sum of the slots.  The first two are one kernel
// that streams the codes of (expert, up to 8 NT of its columns) against those
// columns in shared memory:
//   * Each block makes the plan from the ids itself: the slots in the order of
//     their experts, cut into chunks of nc columns.  The work is chunks x
//     slices of the rows' length x tiles of 16 rows, in that order, and a block
//     takes an even run of it, so that it holds the columns of one or two
//     experts in its lifetime.
//   * A tile is 16 rows for the warp-level tensor instruction m16n8k16: 16 rows
//     of down, or 8 of gate and the same 8 of up.  Codes become exact f16 values
//     in registers; a column is scaled by a power of two into f16's range, in two
//     pieces (22 bits) where its type needs them.  Sums are f32, taken out of the
//     tensor instruction's accumulator, which truncates, every 128 bytes of a row
//     (every 4 of codes where there are two pieces).
//   * A thread copies its own 16 bytes of codes into its own slots of a ring in
//     shared memory (cp.async), several lines ahead and across the tiles of the
//     run: no barrier orders them.  The warps of a block take the 128-byte lines
//     of a tile in turn, or several tiles where rows are short, and add their
//     sums in warp order.
//   * Slices keep a block's columns within shared memory where rows are long or
//     columns many: each slice writes its own sums, the reader adds them in order.
// No sum depends on the order in which blocks run.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "codes_f16.h"
#include "qmat_q8.h"
#include "qwq_internal.h"

namespace qwq {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kPairs = 1024;                  // slots of a launch at most
constexpr int kTokens = 64;                   // tokens of a launch at most
constexpr int kRedPitch = 20;                 // floats of a column's 16 sums in shared memory: no bank conflicts

__device__ unsigned int g_moe_err = 0;        // first error a kernel recorded (a B200Q_E* code, negated)

struct Stream {
    const Expert *table;
    const int *ids;
    const void *x;                            // gate and up: the tokens' rows
    const float *gu;                          // down: the sums of gate and up, [ns_in][P][2][F]
    float *out;                               // gate and up: as gu; down: [ns][P][D]
    long long ldx, ld;                        // values; bytes of a row of codes
    int P, k, E, type, act;                   // P = S * k
    int K, rows, F;                           // columns of the product's rows; its rows (F or D)
    int lines, ns, ns_in;                     // 128-byte lines of a row, slices of them
    int tiles, wk;                            // tiles of the rows; warps that share a tile
    int nc, pitch, B;                         // columns of a chunk, bytes of one in shared memory, where they begin
    bool down;
};

__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_dependents_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------- plan
struct Plan {
    unsigned short order[kPairs];             // slots, by expert
    unsigned short expert[kPairs], first[kPairs];   // of chunk c: its expert, its first place in order
    unsigned char n[kPairs];                  // and its columns
    int count[kMoeMaxExperts];                // slots of an expert, then their first place
    unsigned short rank[kPairs];              // of a slot among its expert's
    short id[kPairs];
    int chunks;
};

__device__ __forceinline__ void make_plan(const Stream &p, Plan &pl) {
    const int tid = threadIdx.x, lane = tid & 31;
    for (int e = tid; e < p.E; e += kThreads) pl.count[e] = 0;
    for (int i = tid; i < p.P; i += kThreads) {
        int e = p.ids[i];
        if (e < -1 || e >= p.E) {
            if (!p.down && blockIdx.x == 0) atomicCAS(&g_moe_err, 0u, (unsigned)(-B200Q_EINVAL));
            e = -1;
        }
        pl.id[i] = (short)e;
    }
    __syncthreads();
    if (tid < 32) {
        // ranks in the order of the slots
        for (int i0 = 0; i0 < p.P; i0 += 32) {
            const int i = i0 + lane, e = i < p.P ? pl.id[i] : -1;
            const unsigned same = __match_any_sync(0xffffffffu, e);
            const int before = e >= 0 ? pl.count[e] : 0;
            __syncwarp();
            if (e >= 0) {
                pl.rank[i] = (unsigned short)(before + __popc(same & ((1u << lane) - 1)));
                if (lane == __ffs(same) - 1) pl.count[e] = before + __popc(same);
            }
            __syncwarp();
        }
        // first places and chunks
        int place = 0, chunk = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane, c = e < p.E ? pl.count[e] : 0, m = (c + p.nc - 1) / p.nc;
            int a = c, b = m;                  // sums up to and with this lane's
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int va = __shfl_up_sync(0xffffffffu, a, o), vb = __shfl_up_sync(0xffffffffu, b, o);
                if (lane >= o) a += va, b += vb;
            }
            const int f = place + a - c;
            if (e < p.E) pl.count[e] = f;
            for (int j = 0; j < m; ++j) {
                const int at = chunk + b - m + j;
                pl.expert[at] = (unsigned short)e;
                pl.first[at] = (unsigned short)(f + j * p.nc);
                pl.n[at] = (unsigned char)min(p.nc, c - j * p.nc);
            }
            place += __shfl_sync(0xffffffffu, a, 31);
            chunk += __shfl_sync(0xffffffffu, b, 31);
        }
        if (lane == 0) pl.chunks = chunk;
    }
    __syncthreads();
    for (int i = tid; i < p.P; i += kThreads)
        if (pl.id[i] >= 0) pl.order[pl.count[pl.id[i]] + pl.rank[i]] = (unsigned short)i;
    __syncthreads();
}

// ---------------------------------------------------------------- columns
// Eight values of a token's row from column c on, 0 past the row.
template <class T> __device__ __forceinline__ float as_float(T v);
template <> __device__ __forceinline__ float as_float<float>(float v) { return v; }
template <> __device__ __forceinline__ float as_float<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float as_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T>
__device__ __forceinline__ void row8(const T *r, int c, int K, float (&v)[8]) {
    union {
        uint4 q[sizeof(T) / 2];
        T e[8];
    } u;
    if (c + 8 <= K && (uintptr_t)(r + c) % 16 == 0) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) u.q[i] = reinterpret_cast<const uint4 *>(r + c)[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = as_float<T>(u.e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < K ? as_float<T>(r[c + i]) : 0.f;
    }
}

// Eight values of column `slot` of the product from column c on: of its token's
// row, or act(gate) * up from the first product's sums.
__device__ __forceinline__ void column8(const Stream &p, int slot, int c, float (&v)[8]) {
    if (!p.down) {
        const long long at = (long long)(slot / p.k) * p.ldx;
        if (p.type == B200Q_T_F32) row8((const float *)p.x + at, c, p.K, v);
        else if (p.type == B200Q_T_F16) row8((const __half *)p.x + at, c, p.K, v);
        else row8((const __nv_bfloat16 *)p.x + at, c, p.K, v);
        return;
    }
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = u[i] = 0.f;
    for (int s = 0; s < p.ns_in; ++s) {
        const float *g = p.gu + ((long long)s * p.P + slot) * 2 * p.F;
        float a[8], b[8];
        row8(g, c, p.F, a);
        row8(g + p.F, c, p.F, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += a[i], u[i] += b[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_q8(v[i], p.act) * u[i];
}

__device__ __forceinline__ uint32_t pack(__half a, __half b) {
    return (uint32_t)__half_as_ushort(a) | (uint32_t)__half_as_ushort(b) << 16;
}

// Eight values to 16 bytes of f16 in the order in which fields() takes a word
// of codes apart, and what is left of them to `rest`.
template <int FMT>
__device__ __forceinline__ void split(const float (&v)[8], float scale, uint4 &hi, uint4 &rest) {
    __half h[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = v[i] * scale;
        h[i] = __float2half_rn(f);
        l[i] = __float2half_rn(f - __half2float(h[i]));
    }
    if constexpr (FMT == B200Q_I4) {           // pairs (0,4) (2,6) (1,5) (3,7)
        hi = make_uint4(pack(h[0], h[4]), pack(h[2], h[6]), pack(h[1], h[5]), pack(h[3], h[7]));
        rest = make_uint4(pack(l[0], l[4]), pack(l[2], l[6]), pack(l[1], l[5]), pack(l[3], l[7]));
    } else {
        hi = make_uint4(pack(h[0], h[1]), pack(h[2], h[3]), pack(h[4], h[5]), pack(h[6], h[7]));
        rest = make_uint4(pack(l[0], l[1]), pack(l[2], l[3]), pack(l[4], l[5]), pack(l[6], l[7]));
    }
}

// The columns of a chunk, lines l0 .. l1-1, into shared memory: per 64 bytes of
// codes and column KC / 8 pieces of 64 bytes, 16 of them for each of the four
// threads that share a row.  unscale[c] is the inverse of column c's scale.
// Called by the whole block; ends with a barrier.
template <int FMT, int PC>
__device__ __forceinline__ void stage(const Stream &p, const unsigned short *order, int n, int l0, int l1, uint8_t *B,
                                      unsigned *top, float *unscale) {
    constexpr int KC = Fmt<FMT>::KC;
    const int units = (l1 - l0) * KC;          // of eight values: KC of them to a line
    const int k0 = l0 * 8 * KC;
    int per = 32;                              // threads per column
    while (per < units && per < kThreads) per *= 2;
    const int sub = threadIdx.x & (per - 1), c0 = threadIdx.x / per, step = kThreads / per;
    for (int c = threadIdx.x; c < n; c += kThreads) top[c] = 0u;
    __syncthreads();
    for (int c = c0; c < n; c += step) {
        unsigned m = 0;
        for (int u = sub; u < units; u += per) {
            float v[8];
            column8(p, order[c], k0 + 8 * u, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if ((threadIdx.x & 31) == 0) atomicMax(&top[c], m);
    }
    __syncthreads();
    for (int c = c0; c < n; c += step) {
        // the largest magnitude to [2^14, 2^15); at most 2^126, so that the inverse is a normal number
        const int up = top[c] ? min(126, 14 + 127 - (int)(top[c] >> 23)) : 0;
        const float scale = __uint_as_float((unsigned)(127 + up) << 23);
        if (sub == 0) unscale[c] = __uint_as_float((unsigned)(127 - up) << 23);
        uint8_t *col = B + c * p.pitch;
        for (int u = sub; u < units; u += per) {
            float v[8];
            uint4 hi, rest;
            int at;
            if constexpr (FMT == B200Q_I2) {
                // a word is 16 codes: the values that its instructions 2j, 2j+1 take, j = u & 1
                const int w = u >> 1, j = u & 1;
                float lo[8], hv[8];
                column8(p, order[c], k0 + 16 * w, lo);
                column8(p, order[c], k0 + 16 * w + 8, hv);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    v[4 * t] = j ? lo[2 + t] : lo[t];
                    v[4 * t + 1] = j ? hv[2 + t] : hv[t];
                    v[4 * t + 2] = j ? lo[6 + t] : lo[4 + t];
                    v[4 * t + 3] = j ? hv[6 + t] : hv[4 + t];
                }
                at = (w >> 4) * 512 + ((w & 3) * 2 + j) * 64 + ((w >> 2) & 3) * 16;
            } else {
                column8(p, order[c], k0 + 8 * u, v);
                constexpr int W = KC / 8;      // units of a thread's 16 bytes of codes
                at = u / (4 * W) * (64 * W) + u % W * 64 + u / W % 4 * 16;
            }
            split<FMT>(v, scale, hi, rest);
            *reinterpret_cast<uint4 *>(col + at) = hi;
            if constexpr (PC == 2) *reinterpret_cast<uint4 *>(col + p.nc * p.pitch + at) = rest;
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- the stream
template <int NT, int MT> struct Shape {
    static constexpr int kAhead = MT == 1 ? 6 : 3;                     // lines in the ring
    static constexpr int kSlot = MT * 2048;                            // bytes of a warp's line
    static constexpr int kRing = kWarps * kAhead * kSlot;
    static constexpr int kRedTile = 8 * NT * kRedPitch;                // floats of a warp's tile
    static constexpr int kRed = kWarps * kRedTile * 4;
    static constexpr int kPlanAt = kRing + kRed + 8 * NT * 8;          // sums, columns' maxima and scales
    static constexpr int kColumns = (kPlanAt + (int)sizeof(Plan) + 127) / 128 * 128;
};

// PC: pieces of a column.
template <int FMT, int NT, int MT, int PC>
__global__ void __launch_bounds__(kThreads, 1) moe_stream_kernel(const __grid_constant__ Stream p) {
    using Sh = Shape<NT, MT>;
    constexpr int KC = Fmt<FMT>::KC, MMAS = Fmt<FMT>::MMAS;
    extern __shared__ __align__(128) uint8_t smem[];
    float *red = reinterpret_cast<float *>(smem + Sh::kRing);
    unsigned *top = reinterpret_cast<unsigned *>(smem + Sh::kRing + Sh::kRed);
    float *unscale = reinterpret_cast<float *>(top + 8 * NT);
    Plan &pl = *reinterpret_cast<Plan *>(smem + Sh::kPlanAt);
    uint8_t *B = smem + Sh::kColumns;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
    const int kw = warp % p.wk, wm = warp / p.wk, groups = kWarps / p.wk;

    // The ids may come from the kernel before gate and up; down follows them, and
    // they were there when gate and up began.
    if (!p.down) dependency_wait();
    make_plan(p, pl);
    const int tile_runs = (p.tiles + groups * MT - 1) / (groups * MT);      // of a slice
    const long long items = (long long)pl.chunks * p.ns * tile_runs;
    const long long lo = items * blockIdx.x / gridDim.x, hi = items * (blockIdx.x + 1) / gridDim.x;

    // the copy cursor: this thread's next line
    long long fitem = lo;
    int fcs = (int)(lo / tile_runs), frun = (int)(lo - (long long)fcs * tile_runs), fchunk = -1, fline = 0, fend = 0, fslot = 0;
    const uint8_t *first = nullptr, *second = nullptr;                      // rows 0-7 and 8-15 of a tile
    long long off[MT];
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (Sh::kAhead * Sh::kSlot) + lane * 16;
    auto open = [&]() {                        // the cursor's item, or a later one that has a line for this warp
        for (; fitem < hi; ++fitem, fcs += ++frun == tile_runs, frun = frun == tile_runs ? 0 : frun) {
            const int c = fcs / p.ns, sl = fcs - c * p.ns, tile = (frun * groups + wm) * MT;
            fline = (int)((long long)sl * p.lines / p.ns) + kw;
            fend = (int)((long long)(sl + 1) * p.lines / p.ns);
            if (fline >= fend || tile >= p.tiles) continue;
            if (c != fchunk) {
                const Expert &e = p.table[pl.expert[c]];
                first = p.down ? e.codes[2] : e.codes[0];
                second = p.down ? e.codes[2] + 8 * p.ld : e.codes[1];
                fchunk = c;
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)       // a tile past the last reads the last again
                off[m] = ((long long)min(tile + m, p.tiles - 1) * (p.down ? 16 : 8) + g) * p.ld + tig * 16;
            return;
        }
    };
    auto copy_line = [&]() {
        if (fitem < hi) {
            const uint32_t to = ring + fslot * Sh::kSlot;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const long long o = off[m] + fline * 128;
                copy16(to + m * 2048, first + o);
                copy16(to + m * 2048 + 512, second + o);
                copy16(to + m * 2048 + 1024, first + o + 64);
                copy16(to + m * 2048 + 1536, second + o + 64);
            }
            if ((fline += p.wk) >= fend) {
                ++fitem;
                if (++frun == tile_runs) frun = 0, ++fcs;
                open();
            }
            if (++fslot == Sh::kAhead) fslot = 0;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");           // empty at the end: the waits count groups
    };
    open();
#pragma unroll 1
    for (int i = 0; i < Sh::kAhead; ++i) copy_line();

    if (p.down) dependency_wait();
    let_dependents_start();

    const uint8_t *slots = smem + warp * (Sh::kAhead * Sh::kSlot) + lane * 16;
    int slot = 0, staged = -1, chunk = -1, n = 0, l0 = 0, l1 = 0, slice = 0;
    const unsigned short *order = nullptr;
    const float *scales = nullptr;
    const int row = tid & 15;                  // of the tile, of the sums that this thread adds
    int cs = (int)(lo / tile_runs), run = (int)(lo - (long long)cs * tile_runs);
    for (long long item = lo; item < hi; ++item) {
        if (cs != staged) {
            __syncthreads();                   // the columns before are read
            const int c = cs / p.ns;
            slice = cs - c * p.ns;
            l0 = (int)((long long)slice * p.lines / p.ns);
            l1 = (int)((long long)(slice + 1) * p.lines / p.ns);
            if (c != chunk) {
                order = pl.order + pl.first[c];
                n = pl.n[c];
                scales = p.table[pl.expert[c]].scales[p.down ? 2 : row < 8 ? 0 : 1];
                chunk = c;
            }
            stage<FMT, PC>(p, order, n, l0, l1, B, top, unscale);
            staged = cs;
        }
        const int tile = (run * groups + wm) * MT;
        float sum[MT][NT][4] = {}, scale[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {         // fetched now, used at the end
            const int o = p.down ? (tile + m) * 16 + row : (tile + m) * 8 + (row & 7);
            scale[m] = o < p.rows ? scales[o] : 0.f;
        }
        if (tile < p.tiles) {
            for (int line = l0 + kw; line < l1; line += p.wk) {
                asm volatile("cp.async.wait_group %0;" ::"n"(Sh::kAhead - 1) : "memory");
                uint4 q[MT][2][2];             // [64 bytes][row half]
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        q[m][i >> 1][i & 1] = *reinterpret_cast<const uint4 *>(slots + slot * Sh::kSlot + m * 2048 + i * 512);
                if (++slot == Sh::kAhead) slot = 0;
                copy_line();                   // into the slot just read: this thread's own
                // sums of this line; two pieces: of a word's first pieces, and of the line's second ones
                float acc[MT][NT][4] = {}, rest[PC == 2 ? MT : 1][PC == 2 ? NT : 1][4] = {};
                const uint8_t *xb = B + (line - l0) * (16 * KC) + tig * 16;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {                      // word of the thread's 16 bytes
                        uint32_t a[MT][MMAS][4];
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const uint4 &c0 = q[m][half][0], &c1 = q[m][half][1];
                            const uint32_t w0 = w == 0 ? c0.x : w == 1 ? c0.y : w == 2 ? c0.z : c0.w;
                            const uint32_t w1 = w == 0 ? c1.x : w == 1 ? c1.y : w == 2 ? c1.z : c1.w;
#pragma unroll
                            for (int t = 0; t < MMAS; ++t) {
                                fields<FMT>(w0, t, a[m][t][0], a[m][t][2]);
                                fields<FMT>(w1, t, a[m][t][1], a[m][t][3]);
                            }
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (NT > 1 && nt * 8 >= n) break;
                            // a column past the chunk's (nc of them are there) is computed and not stored
                            const uint8_t *col = xb + min(nt * 8 + g, p.nc - 1) * p.pitch + half * (8 * KC);
#pragma unroll
                            for (int pc = 0; pc < PC; ++pc) {
                                const uint8_t *from = col + pc * p.nc * p.pitch;
                                auto to = [&](int m) -> float (&)[4] { return pc ? rest[PC == 2 ? m : 0][PC == 2 ? nt : 0] : acc[m][nt]; };
                                if constexpr (MMAS == 1) {
                                    const uint2 b = *reinterpret_cast<const uint2 *>(from + (w >> 1) * 64 + (w & 1) * 8);
#pragma unroll
                                    for (int m = 0; m < MT; ++m)
                                        mma_f16(to(m), a[m][0][0], a[m][0][1], a[m][0][2], a[m][0][3], b.x, b.y);
                                } else {
#pragma unroll
                                    for (int t = 0; t < MMAS; t += 2) {
                                        const uint4 b = *reinterpret_cast<const uint4 *>(from + (w * (MMAS / 2) + t / 2) * 64);
#pragma unroll
                                        for (int m = 0; m < MT; ++m) {
                                            mma_f16(to(m), a[m][t][0], a[m][t][1], a[m][t][2], a[m][t][3], b.x, b.y);
                                            mma_f16(to(m), a[m][t + 1][0], a[m][t + 1][1], a[m][t + 1][2], a[m][t + 1][3], b.z,
                                                    b.w);
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
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sum[m][nt][i] += PC == 2 ? rest[PC == 2 ? m : 0][PC == 2 ? nt : 0][i] : acc[m][nt][i];
            }
        }
        // [column][row] of this warp's part of a tile, added over its warps in order
        auto meet = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + wm), "r"(p.wk * 32) : "memory"); };
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float *mine = red + warp * Sh::kRedTile + 2 * tig * kRedPitch + g;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float *r = mine + nt * 8 * kRedPitch;
                r[0] = sum[m][nt][0], r[kRedPitch] = sum[m][nt][1];
                r[8] = sum[m][nt][2], r[kRedPitch + 8] = sum[m][nt][3];
            }
            meet();
            const int o = p.down ? (tile + m) * 16 + row : (tile + m) * 8 + (row & 7);
            for (int c = (kw * 32 + lane) >> 4; c < n; c += p.wk * 2) {
                const float *r = red + wm * p.wk * Sh::kRedTile + c * kRedPitch + row;
                float v = 0.f;
                for (int w = 0; w < p.wk; ++w) v += r[w * Sh::kRedTile];
                v = v * scale[m] * unscale[c];
                if (o < p.rows) {
                    const long long at = (long long)slice * p.P + order[c];
                    if (p.down) p.out[at * p.rows + o] = v;
                    else p.out[(at * 2 + (row >> 3)) * p.rows + o] = v;
                }
            }
            meet();                            // the sums are read: the next ones may be written
        }
        if (++run == tile_runs) run = 0, ++cs;
    }
}

// ---------------------------------------------------------------- the weighted sum
struct Sum {
    const float *part;                         // [ns][P][D]
    const int *ids;
    const float *wts;
    const void *res;
    void *y;
    long long ldr, ldy;
    int P, k, E, D, ns, type;
};

__global__ void __launch_bounds__(128) moe_sum_kernel(const Sum p) {
    dependency_wait();
    let_dependents_start();
    const long long s = blockIdx.y;
    const int o = blockIdx.x * 128 + threadIdx.x;
    if (o >= p.D) return;
    float y = 0.f;
    for (int j = 0; j < p.k; ++j) {
        const long long at = s * p.k + j;
        const int e = p.ids[at];
        if (e < 0 || e >= p.E) continue;
        float v = 0.f;
        for (int n = 0; n < p.ns; ++n) v += p.part[((long long)n * p.P + at) * p.D + o];
        y = fmaf(p.wts[at], v, y);
    }
    if (p.res) y += load_typed(p.res, s * p.ldr + o, p.type);
    store_typed(p.y, s * p.ldy + o, p.type, y);
}

// ---------------------------------------------------------------- launches
template <class K, class P>
cudaError_t launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, const P &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

// How one of the two products is launched, from its sizes alone.
struct Way {
    int nt, nc, ns, wk, pitch;
    size_t smem;
};

// Columns of a chunk: what an expert has on average and twice its root more, at
// most 8 NT, NT = 1, 2, 4.
int tiles_of_columns(int S, int k, int E) {
    const double avg = (double)S * k / E;
    double root = 1.0;
    while (root * root < avg) root += 0.5;
    const double want = avg + 2.0 * root;
    const int most = (S + 7) / 8;
    const int nt = want <= 8 ? 1 : want <= 16 ? 2 : 4;
    return nt < most ? nt : most >= 4 ? 4 : most >= 2 ? 2 : 1;
}

Way way_of(int fmt, int nt, int pieces, int S, int lines) {
    const int kc = fmt == B200Q_I8 ? 16 : fmt == B200Q_I4 ? 32 : 64;
    Way w{};
    w.nt = nt;
    w.nc = S < 8 * nt ? S : 8 * nt;
    const size_t fixed = nt == 1 ? Shape<1, 1>::kColumns : nt == 2 ? Shape<2, 2>::kColumns : Shape<4, 2>::kColumns;
    const size_t room = 227 * 1024 - fixed;
    for (w.ns = 1; w.ns < lines; ++w.ns) {
        w.pitch = (lines + w.ns - 1) / w.ns * 16 * kc + 64;
        if ((size_t)w.pitch * w.nc * pieces <= room) break;
    }
    const int per = (lines + w.ns - 1) / w.ns;
    w.pitch = per * 16 * kc + 64;
    w.smem = fixed + (size_t)w.pitch * w.nc * pieces;
    w.wk = 1;
    for (int k = kWarps; k > 1; k /= 2)
        if (per >= 2 * k && per * 20 >= (per + k - 1) / k * k * 17) {
            w.wk = k;
            break;
        }
    return w;
}

template <int FMT, int PC>
cudaError_t start(const Stream &p, const Way &w, int grid, cudaStream_t st) {
    auto go = [&](auto kernel) {
        cudaError_t e = allow_dynamic_smem((const void *)kernel, 227 * 1024);
        return e != cudaSuccess ? e : launch(kernel, dim3(grid), kThreads, w.smem, st, p);
    };
    if (w.nt == 1) return go(moe_stream_kernel<FMT, 1, 1, PC>);
    if (w.nt == 2) return go(moe_stream_kernel<FMT, 2, 2, PC>);
    return go(moe_stream_kernel<FMT, 4, 2, PC>);
}

template <int FMT>
cudaError_t run(const Moe &a, cudaStream_t st) {
    const Experts &ex = *a.ex;
    const int part = kPairs / a.k < kTokens ? kPairs / a.k : kTokens;      // tokens per launch
    const int S = a.S < part ? a.S : part, P = S * a.k, b = a.type == B200Q_T_F32 ? 4 : 2;
    const int in_lines = (int)(ex.ld_in / 128), out_lines = (int)(ex.ld_out / 128);
    const int nt = tiles_of_columns(S, a.k, ex.E);
    const int pc_in = a.type == B200Q_T_F32 ? 2 : 1, pc_out = a.type == B200Q_T_BF16 ? 1 : 2;
    const Way wi = way_of(FMT, nt, pc_in, S, in_lines), wo = way_of(FMT, nt, pc_out, S, out_lines);
    const int grid = sm_count(ex.device);
    const size_t n_gu = (size_t)wi.ns * P * 2 * ex.F, n_part = (size_t)wo.ns * P * ex.D;
    float *gu = nullptr;
    cudaError_t e = workspace_alloc((void **)&gu, (n_gu + n_part + 8) * 4, st);
    if (e != cudaSuccess) return e;
    float *sums = gu + (n_gu + 3) / 4 * 4;
    for (int s0 = 0; s0 < a.S && e == cudaSuccess; s0 += part) {
        const int n = a.S - s0 < part ? a.S - s0 : part;
        Stream p{};
        p.table = ex.table;
        p.ids = a.ids + (long long)s0 * a.k;
        p.x = (const char *)a.x + s0 * a.ldx * b;
        p.gu = gu;
        p.out = gu;
        p.ldx = a.ldx;
        p.ld = ex.ld_in;
        p.P = n * a.k;
        p.k = a.k;
        p.E = ex.E;
        p.type = a.type;
        p.act = a.act;
        p.K = ex.D;
        p.rows = p.F = ex.F;
        p.lines = in_lines;
        p.ns = p.ns_in = wi.ns;
        p.tiles = (ex.F + 7) / 8;
        p.wk = wi.wk;
        p.nc = wi.nc;
        p.pitch = wi.pitch;
        e = pc_in == 2 ? start<FMT, 2>(p, wi, grid, st) : start<FMT, 1>(p, wi, grid, st);
        if (e != cudaSuccess) break;
        p.down = true;
        p.out = sums;
        p.ld = ex.ld_out;
        p.K = ex.F;
        p.rows = ex.D;
        p.lines = out_lines;
        p.ns = wo.ns;
        p.tiles = (ex.D + 15) / 16;
        p.wk = wo.wk;
        p.nc = wo.nc;
        p.pitch = wo.pitch;
        e = pc_out == 2 ? start<FMT, 2>(p, wo, grid, st) : start<FMT, 1>(p, wo, grid, st);
        if (e != cudaSuccess) break;
        Sum q{sums, p.ids, a.wts + (long long)s0 * a.k, a.res ? (const char *)a.res + s0 * a.ldr * b : nullptr,
              (char *)a.y + s0 * a.ldy * b, a.ldr, a.ldy, p.P, a.k, ex.E, ex.D, wo.ns, a.type};
        e = launch(moe_sum_kernel, dim3((ex.D + 127) / 128, n), 128, 0, st, q);
    }
    cudaError_t e2 = workspace_free(gu, st);
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
