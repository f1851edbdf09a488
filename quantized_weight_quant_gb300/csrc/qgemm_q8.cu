// 8-bit rows on the fp8 tensor cores: matrix product and gated pair for more
// rows than the few-row kernel takes.
//     D[o, s] = sum_k A[o, k] B[s, k],  A = deq(W) as E4M3, B = the rows' bytes
//     y[s, o] = act(scale[o] xs[s] D + bias[o]) + res[s, o],  or act(g) u
//
// Codes are exact in E4M3: int4 (-8..7) and int2 (-2..1) as one value, int8 as
// the two values 16 * high (signed) and low (0..15), both times 2^-9 so that
// the low field is its own E4M3 byte; B is read as it is.  Products are exact,
// sums are the tensor cores' f32.
//
// Bound: the tensor cores for many rows, the weights' bytes for few; now the
// hand-over between the roles, ~0.4 us per item at N = 176, and the integer work
// of the dequantizers.  In a graph: int4 12288 x 6144 over 1571 rows 110 us, 2150
// TFLOP/s; the pair 207 us, 2290 TFLOP/s (call by call, with one set of weights,
// 221 us); 6144 x 12288 with a residual 112 us (115 us), int8 187 us; int2 5001 x
// 4097 over 77 rows 16.9 us (18.4 us).
//
// Work is cut into (output tile, 128-column k-block) items, tile-major, and
// every CTA takes one contiguous run of them (one CTA per SM at most): whole
// tiles, an equal part of one tile, or even runs that begin and end inside
// tiles, whichever is done first (plan()).  A tile that one CTA holds whole goes
// straight to y; a cut one is written as f32 planes (one per CTA), and the CTA
// whose arrival completes the tile adds the planes in CTA order and runs the
// epilogue, with all its dequantizing and epilogue warps, when its run is done.
// No CTA waits for another, and the order of the additions does not depend on
// the arrivals, so results repeat bit for bit.
//
// Warp roles:
//   warps 0-2  TMA producers: N rows of x8, and the two boxes of 64 code rows
//              (128-byte swizzle for x8; a TMA takes its thread ~160 cycles
//              and an mbarrier test ~290, so one warp for all three copies of
//              an item would be slower than its MMAs);
//   warp 3     issues the MMAs (kind::f8f6f4, 128 x N x 32, A from tensor
//              memory, B from shared memory) into one of two accumulators of up
//              to 192 columns; one commit per item frees both its stage and its
//              A buffer;
//   warps 4 .. dequantizers, three groups of four (int8: two): codes -> E4M3
//              bytes by a 16-entry table lookup in registers (byte permutes),
//              stored to the group's A buffer in tensor memory, natural K order;
//   last four  epilogue.
// The gated pair takes 64 gate and 64 up rows per tile, interleaved by 16 in
// the lanes, so that a gate and its up value sit in one warp, 16 lanes apart.
// Every mbarrier wait is bounded; a wait that gives up records B200Q_ETIMEOUT,
// raises the CTA's abort flag (which ends the other roles' waits), and the CTA
// drains its copies and frees its tensor memory.
#include <cuda.h>

#include <atomic>
#include <cstring>

#include "qmat_q8.h"

namespace qwq {
namespace {

constexpr int BM = 128, BK = 128;
constexpr int kMaxN = 192;                 // rows of x8 per tile
constexpr int kProducers = 3, kWMma = 3, kWDeq = 4;
constexpr int kEpiWarps = 4;
constexpr int kTmemCols = 512, kAccBase = 128, kAccStride = kMaxN;   // A ring: below column 128
constexpr int kSmemLimit = 232448;
constexpr int kSmemFloor = 120 * 1024;      // one CTA per SM: it takes the whole tensor memory
constexpr int kMiscBytes = 512 + 3 * kMaxN * 4;   // barriers and counters, row scales of three tiles
constexpr int kMaxStages = 12;
constexpr long long kWaitNs = 2000000000ll, kDrainNs = kWaitNs / 4;

__device__ unsigned int g_q8_err = 0;
__device__ long long g_q8_wait_ns = kWaitNs;      // limit of the waits; b200q_selftest_q8 shortens it

// PIECES: E4M3 values per code.  CB: code bytes per row and k-block.
// GROUPS: A buffers, and groups of four dequantizing warps (one per tensor-
// memory lane quarter); group g fills buffer g with every GROUPS-th item.  A
// group takes ~1400 cycles per item, most of them waits; three hide that, and
// leave the epilogue the registers that a fourth would take (6144 x 12288 int4
// over 1571 rows with a residual: 163 us with three, 180 us with four).
template <int FMT> struct Fmt;
template <> struct Fmt<B200Q_I8> { static constexpr int PIECES = 2, CB = 128, GROUPS = 2; };
template <> struct Fmt<B200Q_I4> { static constexpr int PIECES = 1, CB = 64, GROUPS = 3; };
template <> struct Fmt<B200Q_I2> { static constexpr int PIECES = 1, CB = 32, GROUPS = 3; };
template <int FMT> struct Roles {
    static constexpr int kWEpi = kWDeq + 4 * Fmt<FMT>::GROUPS;
    static constexpr int kThreads = (kWEpi + kEpiWarps) * 32;
};

// ---------------------------------------------------------------- PTX helpers
__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ unsigned long long global_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ long long wait_limit() { return *(volatile long long *)&g_q8_wait_ns; }

// Waits for a phase; gives up after the limit, or soon after another role has.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    unsigned long long t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if (mbar_test(bar, parity)) return true;
        if ((it & 7) == 7) {
            if (*abort) return false;
            if (t0 == 0) t0 = global_ns();
            else if ((long long)(global_ns() - t0) > wait_limit()) {
                atomicExch(&g_q8_err, (unsigned)(-B200Q_ETIMEOUT));
                *abort = 1;
                return false;
            }
        }
    }
}

// Waits whether or not the CTA is winding down (copies and MMAs in flight must
// finish before it leaves), up to kDrainNs after t0, the start of the role's
// draining.  (A stage that one producer filled and another gave up on never
// completes: its copies land within that time.)
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity, unsigned long long t0) {
    while (!mbar_test(bar, parity) && (long long)(global_ns() - t0) < kDrainNs) {
    }
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}

// One decision for the warp after a wait, and its lanes meet again.
__device__ __forceinline__ bool together(bool ok) { return __all_sync(0xffffffffu, ok) != 0; }

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor: K-major operand, 128-byte swizzle, rows of
// 128 bytes, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr) {
    uint64_t d = 0;
    d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)1 << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// kind::f8f6f4: D f32, A and B E4M3 (format 0), both K-major, M = 128, N = n.
__device__ __forceinline__ uint32_t idesc_e4m3(int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p; }" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}

// tcgen05.ld / st are warp instructions (.sync.aligned): the lanes meet before
// each, since waits and branches of the activations may have parted them.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    __syncwarp();
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    __syncwarp();
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Counters in shared memory for the hand-offs that no copy and no commit is
// part of: release on the add, acquire on the read, CTA scope.  (A test of an
// mbarrier takes several hundred cycles here even when its phase is complete.)
__device__ __forceinline__ void cnt_add(uint32_t addr) {
    asm volatile("red.release.cta.shared::cta.add.u32 [%0], 1;" ::"r"(addr) : "memory");
}

__device__ __forceinline__ uint32_t cnt_read(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ bool cnt_wait(uint32_t addr, uint32_t want, volatile int *abort) {
    unsigned long long t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if ((int)(cnt_read(addr) - want) >= 0) return true;
        if ((it & 255) == 255) {
            if (*abort) return false;
            if (t0 == 0) t0 = global_ns();
            else if ((long long)(global_ns() - t0) > wait_limit()) {
                atomicExch(&g_q8_err, (unsigned)(-B200Q_ETIMEOUT));
                *abort = 1;
                return false;
            }
        }
    }
}

// bar.sync / bar.red are aligned too.
__device__ __forceinline__ void named_sync(int id, int n) {
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// A named barrier that also ORs a predicate over its threads.
__device__ __forceinline__ bool named_sync_or(int id, int n, bool v) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; bar.red.or.pred q, %2, %3, p; selp.u32 %0, 1, 0, q; }"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ unsigned long long cas_acq_rel(unsigned long long *a, unsigned long long cmp,
                                                          unsigned long long val) {
    unsigned long long old;
    asm volatile("atom.acq_rel.gpu.global.cas.b64 %0, [%1], %2, %3;" : "=l"(old) : "l"(a), "l"(cmp), "l"(val)
                 : "memory");
    return old;
}

// ---------------------------------------------------------------- codes -> E4M3
// Four 4-bit fields (the low 16 bits of sel) through a 16-entry byte table:
// entries 0-7 in (a0, a1), 8-15 in (b0, b1).  Two byte permutes on the fields'
// low 3 bits; m, 0xFF where a field's top bit is set, picks between them.
__device__ __forceinline__ uint32_t lut4(uint32_t sel7, uint32_t m, uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1) {
    const uint32_t a = __byte_perm(a0, a1, sel7), b = __byte_perm(b0, b1, sel7);
    return (a & ~m) | (b & m);
}

// prmt in its sign mode (selector bit 3): bytes of 0xFF or 0x00.
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

// E4M3 bytes of 0..7 and of -8..-1.
constexpr uint32_t kPos0 = 0x44403800u, kPos1 = 0x4E4C4A48u, kNeg0 = 0xCACCCED0u, kNeg1 = 0xB8C0C4C8u;

// Eight nibbles of w -> the E4M3 bytes of code - 8, in nibble order.
__device__ __forceinline__ void lut_i4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t s = w & 0x77777777u, w4 = w << 4;
    lo = lut4(s, prmt(w4, w, 0xD9C8u), kNeg0, kNeg1, kPos0, kPos1);
    hi = lut4(s >> 16, prmt(w4, w, 0xFBEAu), kNeg0, kNeg1, kPos0, kPos1);
}

// Sixteen 2-bit codes -> sixteen E4M3 bytes of code - 2.
__device__ __forceinline__ void lut_i2(uint32_t w, uint32_t *o) {
    constexpr uint32_t t = 0x3800B8C0u;      // -2, -1, 0, 1
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t x = h ? w >> 16 : w & 0xFFFFu;         // 8 codes, spread to one per nibble
        x = (x | (x << 8)) & 0x00FF00FFu;
        x = (x | (x << 4)) & 0x0F0F0F0Fu;
        x = (x | (x << 2)) & 0x33333333u;
        o[2 * h] = __byte_perm(t, 0u, x);
        o[2 * h + 1] = __byte_perm(t, 0u, x >> 16);
    }
}

// The 64 codes of half a row's k-block -> 16 registers per piece.
template <int FMT>
__device__ __forceinline__ void dequant(uint32_t c_s, int row, int half, uint32_t (&p0)[16], uint32_t (&p1)[16]) {
    constexpr int CB = Fmt<FMT>::CB, kChunks = CB / 32;      // 16-byte chunks per half row
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        const int c = half * kChunks + j;
        // the TMA swizzle of rows of CB bytes: chunk index xor bits of the row
        const int pc = CB == 128 ? c ^ (row & 7) : CB == 64 ? c ^ ((row >> 1) & 3) : c ^ ((row >> 2) & 1);
        uint4 q;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                     : "r"(c_s + row * CB + pc * 16)
                     : "memory");
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (FMT == B200Q_I4) {
                lut_i4(w[k], p0[8 * j + 2 * k], p0[8 * j + 2 * k + 1]);
            } else if constexpr (FMT == B200Q_I2) {
                lut_i2(w[k], &p0[4 * k]);
            } else {
                // high nibbles: 16 h 2^-9 = h 2^-5 through the table; low nibbles: l 2^-9 is the byte l
                const uint32_t h = (w[k] >> 4) & 0x0F0F0F0Fu, t = h | (h >> 4);
                const uint32_t f = __byte_perm(t, 0u, 0x4420u);                    // four fields in 16 bits
                const uint32_t f4 = f << 4;
                const uint32_t m = prmt(f4, f, 0xD9C8u);
                constexpr uint32_t d = 0x28282828u;
                p0[4 * j + k] = lut4(f & 0x7777u, m, kPos0 - 0x28282800u, kPos1 - d, kNeg0 - d, kNeg1 - d);
                p1[4 * j + k] = w[k] & 0x0F0F0F0Fu;
            }
        }
    }
}

// ---------------------------------------------------------------- kernel
struct Q8Params {
    const float *scale_g, *scale_u, *bias_g, *bias_u, *xs;
    const void *res;
    void *y;
    long long ldr, ldy;
    float *planes;                 // [grid][2][N][128]
    unsigned long long *cnt;       // [tiles] (token << 10) | arrivals; any other tag counts as no arrivals
    unsigned long long token;
    int O, S, N, nk, n_tiles, act, type;
    int stages;
    int items;                     // tiles * nk
    int grain;                     // a CTA's run is a multiple of this many items: 1, or nk (whole tiles)
};

__device__ __forceinline__ int run_start(const Q8Params &p, int c) {
    return (int)((long long)c * (p.items / p.grain) / (long long)gridDim.x) * p.grain;
}
__device__ __forceinline__ int owner_of(const Q8Params &p, int i) {
    return (int)(((i + 1ll) * (long long)gridDim.x - 1) / p.items);
}

// One more CTA has written its plane of a cut tile; true for the last.
__device__ __forceinline__ bool arrive(const Q8Params &p, int tile) {
    const int t0 = tile * p.nk, pieces = owner_of(p, t0 + p.nk - 1) - owner_of(p, t0) + 1;
    const unsigned long long tag = p.token << 10;
    unsigned long long old = *(volatile unsigned long long *)&p.cnt[tile];
    for (;;) {
        const int n = (old >> 10) == p.token ? (int)(old & 1023) + 1 : 1;
        const unsigned long long prev = cas_acq_rel(&p.cnt[tile], old, n == pieces ? 0ull : tag | (unsigned)n);
        if (prev == old) return n == pieces;
        old = prev;
    }
}

// A CTA that gave up arrives at its cut tiles from item i on all the same, with
// nothing written: their outputs are lost, which the status says, but every
// count is back at 0 when the launch ends.  (A count that stayed would go on
// under the same tag in a captured launch's next replay, and complete its tile
// before the planes are there.)
__device__ __forceinline__ void arrive_rest(const Q8Params &p, int i, int i1) {
    if (!p.planes) return;
    while (i < i1) {
        const int tile = i / p.nk, t0 = tile * p.nk, end = min(t0 + p.nk, i1);
        if (i != t0 || end != t0 + p.nk) arrive(p, tile);
        i = end;
    }
}

template <class T> __device__ __forceinline__ T narrow(float v);
template <> __device__ __forceinline__ float narrow<float>(float v) { return v; }
template <> __device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The bits of eight residual values of this lane's output, tokens s0 .. s0 + 7.
// Read a batch ahead (12288 x 6144 over 1571 rows: 183 us with the reads after
// a batch's arithmetic, 143 us before it, 119 us a batch ahead); past the last
// token or output a value that exists is read instead, so that no load is
// under a branch.
__device__ __forceinline__ void load_res(const Q8Params &p, uint32_t (&rv)[8], int s0, int last, int o) {
    if (!p.res) return;
    const int oc = min(o, p.O - 1);
    if (p.type == B200Q_T_F32) {
#pragma unroll
        for (int k = 0; k < 8; ++k) rv[k] = __ldcg((const unsigned *)p.res + min(s0 + k, last) * p.ldr + oc);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) rv[k] = __ldcg((const unsigned short *)p.res + min(s0 + k, last) * p.ldr + oc);
    }
}

template <class T> __device__ __forceinline__ float widen(uint32_t bits);
template <> __device__ __forceinline__ float widen<float>(uint32_t bits) { return __uint_as_float(bits); }
template <> __device__ __forceinline__ float widen<__half>(uint32_t bits) {
    return __half2float(__ushort_as_half((unsigned short)bits));
}
template <> __device__ __forceinline__ float widen<__nv_bfloat16>(uint32_t bits) {
    return __bfloat162float(__ushort_as_bfloat16((unsigned short)bits));
}

// Eight values: v += res, then y, for tokens s0, s0 + step, ... below s0 + left.
template <class T, int W>
__device__ __forceinline__ void put8(const Q8Params &p, float (&v)[W], const uint32_t (&rv)[8], int s0, int step,
                                     int left, int o) {
    if (p.res) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += widen<T>(rv[k]);
    }
    T *y = (T *)p.y + s0 * p.ldy + o;
    const long long d = step * p.ldy;
#pragma unroll
    for (int k = 0; k < 8; ++k, y += d)
        if (step * k < left) *y = narrow<T>(v[k]);
}

// W accumulator columns (tokens s0 ..; left: how many exist) of this lane's row
// -> eight values of y.  The product takes 8 columns.  The pair takes 16: lanes
// 0-15 hold gate rows, lanes 16-31 the up rows of the same outputs; of two
// neighbouring columns the lower lane finishes the first and the upper lane the
// second, one shuffle for both.
template <bool GLU, int W>
__device__ __forceinline__ void finish(const Q8Params &p, float (&v)[W], const uint32_t (&rv)[8], const float *xs,
                                       float sc, float b, int s0, int left, int o, bool live, bool up) {
    static_assert(W == (GLU ? 16 : 8), "columns");
#pragma unroll
    for (int j = 0; j < W; j += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(xs + j);
        v[j] = fmaf(v[j], x.x * sc, b);
        v[j + 1] = fmaf(v[j + 1], x.y * sc, b);
        v[j + 2] = fmaf(v[j + 2], x.z * sc, b);
        v[j + 3] = fmaf(v[j + 3], x.w * sc, b);
    }
    float u[8];
    if constexpr (GLU) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float got = __shfl_xor_sync(0xffffffffu, up ? v[2 * j] : v[2 * j + 1], 16);
            u[j] = up ? v[2 * j + 1] : got;
            v[j] = up ? got : v[2 * j];
        }
        s0 += up, left -= up;
    }
    switch (p.act) {
    case B200Q_ACT_RELU: act_n<B200Q_ACT_RELU, 8>(v); break;
    case B200Q_ACT_GELU: act_n<B200Q_ACT_GELU, 8>(v); break;
    case B200Q_ACT_GELU_TANH: act_n<B200Q_ACT_GELU_TANH, 8>(v); break;
    case B200Q_ACT_SILU: act_n<B200Q_ACT_SILU, 8>(v); break;
    }
    if constexpr (GLU) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= u[j];
    }
    if (!live) return;
    if (p.type == B200Q_T_F32) put8<float>(p, v, rv, s0, GLU ? 2 : 1, left, o);
    else if (p.type == B200Q_T_F16) put8<__half>(p, v, rv, s0, GLU ? 2 : 1, left, o);
    else put8<__nv_bfloat16>(p, v, rv, s0, GLU ? 2 : 1, left, o);
}

// What a lane of an output tile's epilogue works on.
template <int FMT, bool GLU> struct Outs {
    int tok0, ns, o;               // first row of x8 and how many; output
    bool live, up;
    float sc, b;
    __device__ __forceinline__ Outs(const Q8Params &p, int tile, int quarter, int lane) {
        const int mt = tile / p.n_tiles;
        tok0 = (tile - mt * p.n_tiles) * p.N;
        ns = p.S - tok0 < p.N ? p.S - tok0 : p.N;
        o = GLU ? mt * 64 + quarter * 16 + (lane & 15) : mt * 128 + quarter * 32 + lane;
        live = o < p.O;
        up = GLU && lane >= 16;
        const float unit = FMT == B200Q_I8 ? 512.f : 1.f;      // int8 values are times 2^-9
        sc = live ? (up ? p.scale_u[o] : p.scale_g[o]) * unit : 0.f;
        const float *bias = up ? p.bias_u : p.bias_g;
        b = live && bias ? bias[o] : 0.f;
    }
};

// A cut tile: its CTAs' planes added in CTA order, and the epilogue, by `groups`
// groups of four warps of which this is group g.  32 loads of a thread are in
// flight at a time, also where a tile has fewer planes than that takes (absent
// ones count as 0).
template <int FMT, bool GLU>
__device__ __forceinline__ void add_planes(const Q8Params &p, int tile, const float *xs, int g, int groups) {
    constexpr int W = GLU ? 16 : 8, Z = 32 / W;
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    const Outs<FMT, GLU> r(p, tile, quarter, lane);
    const int t0 = tile * p.nk, first_c = owner_of(p, t0), pieces = owner_of(p, t0 + p.nk - 1) - first_c + 1;
    const long long plane = (long long)p.N * BM;
    const float *planes = p.planes + quarter * 32 + lane + (long long)first_c * 2 * plane;
    // only a tile's first CTA can hold it in its second plane
    const long long pl0 = run_start(p, first_c) / p.nk == tile ? 0 : plane;
    for (int c = g * W; c < r.ns; c += groups * W) {
        uint32_t rv[8];
        if (!GLU) load_res(p, rv, r.tok0 + c, r.tok0 + r.ns - 1, r.o);
        float v[W];
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = 0.f;
        for (int z0 = 0; z0 < pieces; z0 += Z) {
            float q[Z][W];
#pragma unroll
            for (int z = 0; z < Z; ++z) {
                const float *pz = planes + (z0 + z ? (z0 + z) * 2 * plane : pl0) + c * BM;
#pragma unroll
                for (int j = 0; j < W; ++j) q[z][j] = z0 + z < pieces ? __ldcg(pz + j * BM) : 0.f;
            }
#pragma unroll
            for (int z = 0; z < Z; ++z)
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] += q[z][j];
        }
        finish<GLU>(p, v, rv, xs + c, r.sc, r.b, r.tok0 + c, r.ns - c, r.o, r.live, r.up);
    }
}

template <int FMT, bool GLU>
__global__ void __launch_bounds__(Roles<FMT>::kThreads, 1)
    qgemm_q8_kernel(const __grid_constant__ CUtensorMap map_g, const __grid_constant__ CUtensorMap map_u,
                    const __grid_constant__ CUtensorMap map_x, const __grid_constant__ Q8Params p) {
    constexpr int PIECES = Fmt<FMT>::PIECES, CB = Fmt<FMT>::CB, C_BYTES = BM * CB;
    constexpr int kACols = 32 * PIECES, kNumA = Fmt<FMT>::GROUPS, kWEpi = Roles<FMT>::kWEpi;
    static_assert(kACols * kNumA <= kAccBase, "A ring");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const int b_bytes = p.N * BK, kStages = p.stages;
    uint8_t *b_s = smem;                                  // [stages][N][128], 128-byte swizzle
    uint8_t *c_s = b_s + kStages * b_bytes;               // [stages][128][CB], CB-byte swizzle
    float *xs_s = reinterpret_cast<float *>(c_s + kStages * C_BYTES);      // [3][kMaxN] row scales of a tile
    uint64_t *bars = reinterpret_cast<uint64_t *>(xs_s + 3 * kMaxN);
    uint64_t *full = bars, *done = bars + kMaxStages;      // per stage: copies landed; MMAs finished
    uint64_t *acc_full = done + kMaxStages, *acc_empty = acc_full + 2;
    uint32_t *a_ready = reinterpret_cast<uint32_t *>(acc_empty + 2);       // [4] warps that have filled A buffer g, counted on
    uint64_t *fin = reinterpret_cast<uint64_t *>(a_ready + 4);             // after the last MMA
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(fin + 1);
    volatile int *abort = reinterpret_cast<int *>(tmem_slot + 1);
    volatile int *completed = abort + 1;                   // [2] this CTA was the last to arrive at its first, last tile

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: uniform
    const int i0 = run_start(p, blockIdx.x), i1 = run_start(p, blockIdx.x + 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&full[s]), kProducers);
            mbar_init(smem_u32(&done[s]), 1);
        }
        for (int s = 0; s < kNumA; ++s) a_ready[s] = 0;
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&acc_full[b]), 1);
            mbar_init(smem_u32(&acc_empty[b]), kEpiWarps);
        }
        mbar_init(smem_u32(fin), 1);
        *abort = 0;
        completed[0] = completed[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kWMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // all columns are this CTA's, so they start at 0; anything else would be addressed wrongly below
    constexpr uint32_t tmem_base = 0;
    if (*tmem_slot != tmem_base) {
        if (threadIdx.x == 0) {
            atomicExch(&g_q8_err, (unsigned)(-B200Q_ECUDA));
            arrive_rest(p, i0, i1);
        }
        __syncthreads();
        if (warp == kWMma)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*tmem_slot), "r"(kTmemCols)
                         : "memory");
        return;
    }

    if (warp < kProducers) {
        // ---------------- TMA producers: warp 0 the rows of x8, warps 1 and 2 a box of codes each.
        // The whole warp walks the items (so that addresses stay in uniform registers), one lane issues.
        const bool leader = elect_one();
        const uint32_t bytes = warp == 0 ? (uint32_t)b_bytes : (uint32_t)(C_BYTES / 2);
        const CUtensorMap *map = warp == 0 ? &map_x : GLU && warp == 2 ? &map_u : &map_g;
        const uint32_t dst0 = warp == 0 ? smem_u32(b_s) : smem_u32(c_s + (warp - 1) * (C_BYTES / 2));
        const uint32_t step = warp == 0 ? (uint32_t)b_bytes : (uint32_t)C_BYTES;
        const int kcols = warp == 0 ? BK : CB;
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        int tile = i0 / p.nk, kb = i0 % p.nk;
        int mt = tile / p.n_tiles, nt = tile - mt * p.n_tiles;
        const int n = i1 - i0;
        for (int i = 0; i < n; ++i) {
            if (!together(mbar_wait(smem_u32(&done[stage]), phase ^ 1, abort))) break;
            const uint32_t bar = smem_u32(&full[stage]);
            const int row = warp == 0 ? nt * p.N : GLU ? mt * 64 : mt * 128 + (warp - 1) * 64;
            if (leader) {
                mbar_expect_tx(bar, bytes);
                tma_load_2d(dst0 + stage * step, map, kb * kcols, row, bar);
            }
            ++issued;
            if (++stage == kStages) stage = 0, phase ^= 1;
            if (++kb == p.nk) {
                kb = 0;
                if (++nt == p.n_tiles) nt = 0, ++mt;
            }
        }
        __syncwarp();
        // the last copies land before the CTA may leave (a completed phase returns at once)
        const unsigned long long t0 = global_ns();
        for (int k = issued < kStages ? 0 : issued - kStages; k < issued; ++k)
            mbar_drain(smem_u32(&full[k % kStages]), (uint32_t)((k / kStages) & 1), t0);
    } else if (warp == kWMma) {
        // ---------------- MMA issuer: the whole warp walks the items, one lane issues
        const bool leader = elect_one();
        const uint32_t idesc = idesc_e4m3(p.N);
        const uint64_t desc0 = sw128_desc(smem_u32(b_s));
        int stage = 0, abuf = 0, t = 0;
        uint32_t phase = 0, ready = 4;
        int kb = i0 % p.nk;
        bool first = true;
        uint32_t d_tmem = 0;
        uint32_t seen = cnt_read(smem_u32(&a_ready[0]));
        const int n = i1 - i0;
        for (int i = 0; i < n; ++i) {
            if (first) {
                if (!together(mbar_wait(smem_u32(&acc_empty[t & 1]), ((t >> 1) & 1) ^ 1, abort))) break;
                d_tmem = tmem_base + kAccBase + (t & 1) * kAccStride;
            }
            // the dequantizers arrive only after the item's copies have landed
            if (!together((int)(seen - ready) >= 0 || cnt_wait(smem_u32(&a_ready[abuf]), ready, abort))) break;
            tc_fence_after();
            const uint32_t a_tmem = tmem_base + abuf * kACols;
            const uint64_t desc = desc0 + (uint64_t)((stage * b_bytes) >> 4);
            if (++abuf == kNumA) abuf = 0, ready += 4;
            seen = cnt_read(smem_u32(&a_ready[abuf]));      // the next item's, its latency under these MMAs
            const bool last = ++kb == p.nk || i + 1 == n;
            if (leader) {
#pragma unroll
                for (int k = 0; k < BK / 32; ++k)
#pragma unroll
                    for (int pc = 0; pc < PIECES; ++pc)
                        mma_f8(d_tmem, a_tmem + 32 * pc + 8 * k, desc + 2 * k, idesc,
                               (first && k == 0 && pc == 0) ? 0u : 1u);
                mma_commit(smem_u32(&done[stage]));
                if (last) mma_commit(smem_u32(&acc_full[t & 1]));
            }
            first = last;
            if (last) kb = 0, ++t;
            if (++stage == kStages) stage = 0, phase ^= 1;
        }
        // everything issued, also before giving up, and its arrivals in shared memory land before the CTA may leave
        __syncwarp();
        if (leader) mma_commit(smem_u32(fin));
        mbar_drain(smem_u32(fin), 0, global_ns());
    } else if (warp < kWEpi) {
        // ---------------- dequantizers: group g, items g, g + GROUPS, ..., one thread per row
        const int quarter = warp & 3, g = (warp - kWDeq) >> 2;
        // shared-memory row of this thread's lane (the pair: 16 gate rows, then 16 up rows per quarter)
        const int row = GLU ? (lane >> 4) * 64 + quarter * 16 + (lane & 15) : quarter * 32 + lane;
        const uint32_t tdst = tmem_base + ((uint32_t)(quarter * 32) << 16) + g * kACols;
        int stage = g, fstage = 0;                 // the item's stage; the stage of the buffer's previous item
        uint32_t phase = 0, fphase = 0;
        for (int i = i0 + g; i < i1; i += kNumA) {
            if (!together(mbar_wait(smem_u32(&full[stage]), phase, abort))) break;
            uint32_t v0[16], v1[16];
            dequant<FMT>(smem_u32(c_s) + stage * C_BYTES, row, 0, v0, v1);
            // the buffer is free when the MMAs of its previous item have finished (the barrier cannot
            // run a phase ahead: that takes this item, as kStages >= kNumA)
            if (i >= i0 + kNumA && !together(mbar_wait(smem_u32(&done[fstage]), fphase, abort))) break;
            tc_fence_after();
            tmem_st16(tdst, v0);
            if (PIECES == 2) tmem_st16(tdst + 32, v1);
            dequant<FMT>(smem_u32(c_s) + stage * C_BYTES, row, 1, v0, v1);
            tmem_st16(tdst + 16, v0);
            if (PIECES == 2) tmem_st16(tdst + 48, v1);
            __syncwarp();
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) cnt_add(smem_u32(&a_ready[g]));
            fstage = stage, fphase = phase;
            stage += kNumA;
            if (stage >= kStages) stage -= kStages, phase ^= 1;
        }
    } else {
        // ---------------- epilogue: tensor-memory lanes 32 * (warp % 4) .., W columns at a time
        constexpr int kEpi = kEpiWarps * 32, W = GLU ? 16 : 8;
        const int quarter = warp & 3, et = threadIdx.x - kWEpi * 32;
        const int arow = quarter * 32 + lane;
        int t = 0, i = i0;
        for (; i < i1; ++t) {
            const int tile = i / p.nk, t0 = tile * p.nk, t1 = t0 + p.nk;
            const int end = min(t1, i1);
            const bool whole = i == t0 && end == t1;
            // the tile's scales and bias, while its MMAs run
            const Outs<FMT, GLU> r(p, tile, quarter, lane);
            float *xs = xs_s + (t ? t & 1 : 2) * kMaxN;       // the first tile's stay for the end
            for (int c = et; c < p.N; c += kEpi) xs[c] = c < r.ns ? p.xs[r.tok0 + c] : 0.f;
            // the residual's lines into L2 while the MMAs run (64 bytes per row and warp)
            if (p.res && whole) {
                const int ob = p.type == B200Q_T_F32 ? 4 : 2, o0 = r.o - lane;
                if (o0 < p.O)
                    for (int c = lane; c < r.ns; c += 32)
                        asm volatile(
                            "prefetch.global.L2 [%0];" ::"l"((const char *)p.res + ((r.tok0 + c) * p.ldr + o0) * ob));
            }
            // one decision for the four warps, and xs is written
            if (named_sync_or(1, kEpi, !mbar_wait(smem_u32(&acc_full[t & 1]), (t >> 1) & 1, abort))) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + kAccBase + (t & 1) * kAccStride;
            if (whole) {
                uint32_t next[8];
                if (!GLU) load_res(p, next, r.tok0, r.tok0 + r.ns - 1, r.o);
                for (int c = 0; c < r.ns; c += W) {
                    uint32_t rv[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) rv[j] = next[j];
                    if (!GLU) load_res(p, next, r.tok0 + c + W, r.tok0 + r.ns - 1, r.o);
                    float v[W];
                    tmem_ld(taddr + c, v);
                    finish<GLU>(p, v, rv, xs + c, r.sc, r.b, r.tok0 + c, r.ns - c, r.o, r.live, r.up);
                }
            } else {
                // this CTA's plane, [N][128 rows], then the tile's arrival count
                float *pl = p.planes + ((long long)blockIdx.x * 2 + (i == i0 ? 0 : 1)) * p.N * BM + arow;
                for (int c = 0; c < p.N; c += W) {
                    float v[W];
                    tmem_ld(taddr + c, v);
#pragma unroll
                    for (int j = 0; j < W; ++j) pl[(c + j) * BM] = v[j];
                }
                named_sync(1, kEpi);
                if (et == 0) completed[t != 0] = arrive(p, tile);      // only a CTA's first and last tiles are cut
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&acc_empty[t & 1]));
            i = end;
        }
        if (et == 0) arrive_rest(p, i, i1);
    }

    // Cut tiles that this CTA completed, with the dequantizers' help (their work is done): 176 rows of
    // 6144 x 12288 with a residual, three planes per tile: 51 us by the epilogue warps alone, 30 us by all.
    if (p.planes && warp >= kWDeq) {
        named_sync(2, (kWEpi + kEpiWarps - kWDeq) * 32);
        for (int k = 0; k < 2; ++k) {
            if (!completed[k]) continue;
            const int t = k ? (i1 - 1) / p.nk - i0 / p.nk : 0;
            add_planes<FMT, GLU>(p, i0 / p.nk + t, xs_s + (t ? t & 1 : 2) * kMaxN, (warp - kWDeq) >> 2, kNumA + 1);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols)
                     : "memory");
}

// A launch's 54-bit tag: every launch its own, and spread over all bits (the
// finalizer of splitmix64: G. Steele, D. Lea, C. Flood, "Fast splittable
// pseudorandom number generators", 2014), so that what an earlier use left in
// the workspace does not look like one.  A count returns to 0 when all of its
// tile's CTAs have arrived, which those that give up do too, so a captured
// launch finds no count of its last replay.
unsigned long long next_token() {
    static std::atomic<unsigned long long> launches{0};
    unsigned long long z = (launches.fetch_add(1, std::memory_order_relaxed) + 1) * 0x9E3779B97F4A7C15ull;
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return (z ^ (z >> 31)) >> 10;
}

template <int FMT, bool GLU>
GemmPlan plan(int O, int I, int S, int n_sms) {
    constexpr int C_BYTES = BM * Fmt<FMT>::CB;
    GemmPlan r{};
    // rows of x8 per tile: the fewest tiles of at most kMaxN rows, evenly filled
    const int n_tiles = (int)((S + (kMaxN - 1ll)) / kMaxN);
    const int N = r.N = (int)(((S + (n_tiles - 1ll)) / n_tiles + 15) / 16 * 16);
    const int nk = r.nk = (int)((I + (BK - 1ll)) / BK);
    r.n_tiles = (int)((S + (N - 1ll)) / N);
    const long long m_tiles = GLU ? (O + 63ll) / 64 : (O + 127ll) / 128;
    const long long tiles = r.tiles = m_tiles * r.n_tiles;
    if (tiles * nk > 0x7ffffff0ll) return r;
    r.items = (int)(tiles * nk);
    // Three ways to share the items out.  Counted is what the busiest CTA has to
    // do, in items, and for the planes and the join 12 items with one shared tile
    // and 17 + N / 16 with two (int8, whose items take longer, three quarters of
    // that and 11).  Fitted to 714 calls timed in every form, 512 to 19456 outputs,
    // 512 to 12288 columns, 16 to 512 rows: the form taken is 0.3 % slower than the
    // fastest on average, 9 % at most.
    const int one_shared = FMT == B200Q_I8 ? 11 : 12, two_shared = (17 + N / 16) * (FMT == B200Q_I8 ? 3 : 4) / 4;
    // Whole tiles, with an uneven last round (6144 x 12288 over 1571 rows with a
    // residual, 288 items instead of 273: 113 us, 120 us in even runs; int4 12288 x
    // 256 over 176 rows, 96 CTAs: 11.7 us, 33.0 us in runs of eight items).
    long long grid = tiles < n_sms ? tiles : n_sms;
    long long least = (tiles + grid - 1) / grid * nk;
    bool even = true;
    // Few tiles: the same number of CTAs for every tile, each with one part of
    // one tile, of eight items at least (int2 5001 x 4097 over 77 rows, three
    // CTAs a tile: 16.9 us, 20.8 us in even runs over all SMs).
    const long long k = n_sms / tiles;
    if (k > 1 && nk / k >= 8 && (nk + k - 1) / k + one_shared < least) {
        least = (nk + k - 1) / k + one_shared;
        grid = tiles * k;
        even = false;
    }
    // Even runs over all SMs, of eight items at least, with a shared tile at both
    // ends (int4 10240 x 12288 over 16 rows, 51 items instead of 96: 26.5 us, 34.7
    // us with 80 whole tiles; int8 8192 x 8192 over 32 rows, 27 items instead of
    // 32: 27.8 us, 29.5 us with two CTAs a tile; the other way round the pair 5120
    // x 6144 over 192 rows, 31.8 us, and 26.5 us whole).
    const long long runs = r.items < 8ll * n_sms ? (r.items + 7ll) / 8 : n_sms;
    if ((r.items + runs - 1) / runs + two_shared < least) {
        grid = runs;
        even = false;
    }
    r.grid = (int)grid;
    r.grain = even ? nk : 1;
    r.cut = !even && (r.items % grid != 0 || (r.items / grid) % nk != 0);
    r.plane_bytes = r.cut ? grid * 2 * N * BM * 4 : 0;
    const int per = N * BK + C_BYTES;
    r.stages = (kSmemLimit - 1024 - kMiscBytes) / per;
    if (r.stages > kMaxStages) r.stages = kMaxStages;
    r.smem = 1024 + (size_t)r.stages * per + kMiscBytes;
    if (r.smem < kSmemFloor) r.smem = kSmemFloor;
    r.ok = true;
    return r;
}

template <int FMT, bool GLU>
cudaError_t run(const MatQ8 &a, cudaStream_t st) {
    const Tensor &t = *a.tg;
    const GemmPlan r = plan<FMT, GLU>(t.O, t.I, a.S, sm_count(t.device));
    if (!r.ok) return cudaErrorInvalidValue;
    CUtensorMap map_x;
    if (!tmap_encode_2d(&map_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x8, (uint64_t)t.I, (uint64_t)a.S, (uint64_t)a.ld8, BK,
                        (uint32_t)r.N, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    Q8Params p{};
    p.scale_g = t.scales;
    p.scale_u = a.tu ? a.tu->scales : nullptr;
    p.bias_g = a.bias_g;
    p.bias_u = a.bias_u;
    p.xs = a.xs;
    p.res = a.res;
    p.y = a.y;
    p.ldr = a.ldr;
    p.ldy = a.ldy;
    p.O = t.O;
    p.S = a.S;
    p.N = r.N;
    p.nk = r.nk;
    p.n_tiles = r.n_tiles;
    p.act = a.act;
    p.type = a.type;
    p.items = r.items;
    p.grain = r.grain;
    p.stages = r.stages;
    cudaError_t e = allow_dynamic_smem((const void *)qgemm_q8_kernel<FMT, GLU>, kSmemLimit);
    if (e != cudaSuccess) return e;
    void *ws = nullptr;
    if (r.cut) {
        e = workspace_alloc(&ws, (size_t)r.plane_bytes + (size_t)r.tiles * 8, st);
        if (e != cudaSuccess) return e;
        p.planes = (float *)ws;
        p.cnt = (unsigned long long *)((char *)ws + r.plane_bytes);
        p.token = next_token();
    }
    qgemm_q8_kernel<FMT, GLU><<<r.grid, Roles<FMT>::kThreads, r.smem, st>>>(t.q8_map, a.tu ? a.tu->q8_map : t.q8_map, map_x, p);
    count_launch();
    e = cudaGetLastError();
    if (ws) {
        const cudaError_t ef = workspace_free(ws, st);
        if (e == cudaSuccess) e = ef;
    }
    return e;
}

}  // namespace

// Codes as bytes [o_pad, ld], box 64 rows x one k-block, swizzled by the
// box's width so that the dequantizers' 16-byte reads touch every bank once.
bool q8_map_encode(Tensor &t) {
    memset(&t.q8_map, 0, sizeof t.q8_map);
    if (fmt_bits(t.fmt) == 0 || t.fmt == B200Q_F32) return true;
    const uint32_t cb = t.fmt == B200Q_I8 ? 128 : t.fmt == B200Q_I4 ? 64 : 32;
    return tmap_encode_2d(&t.q8_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, t.codes, (uint64_t)t.ld, (uint64_t)t.o_pad,
                          (uint64_t)t.ld, cb, 64,
                          cb == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                          : cb == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                     : CU_TENSOR_MAP_SWIZZLE_32B);
}

GemmPlan plan_gemm_q8(int fmt, bool pair, int O, int I, int S, int n_sms) {
    switch (fmt) {
    case B200Q_I8: return pair ? plan<B200Q_I8, true>(O, I, S, n_sms) : plan<B200Q_I8, false>(O, I, S, n_sms);
    case B200Q_I4: return pair ? plan<B200Q_I4, true>(O, I, S, n_sms) : plan<B200Q_I4, false>(O, I, S, n_sms);
    case B200Q_I2: return pair ? plan<B200Q_I2, true>(O, I, S, n_sms) : plan<B200Q_I2, false>(O, I, S, n_sms);
    }
    return GemmPlan{};
}

// Item numbers are 32-bit: longer batches in parts of at most 2^16 rows, fewer for a large tensor.
int gemm_q8_part(int O, int I) {
    const long long row_items = ((O + 63ll) / 64) * ((I + (BK - 1ll)) / BK);
    int part = 1 << 16;
    while (part > 128 && row_items * ((part + kMaxN - 1) / kMaxN) > 0x7ffffff0ll) part /= 2;
    return part;
}

int gemm_q8_parts(int S, int part) { return (int)((S + (part - 1ll)) / part); }

cudaError_t launch_gemm_q8(const MatQ8 &a, cudaStream_t st) {
    const int part = gemm_q8_part(a.tg->O, a.tg->I);
    const long long b = a.type == B200Q_T_F32 ? 4 : 2;
    const int parts = gemm_q8_parts(a.S, part);
    for (int k = 0; k < parts; ++k) {
        const long long s0 = (long long)k * part;
        MatQ8 c = a;
        c.S = (int)(a.S - s0 < part ? a.S - s0 : part);
        c.x8 += s0 * a.ld8;
        c.xs += s0;
        c.y = (char *)a.y + s0 * a.ldy * b;
        if (a.res) c.res = (const char *)a.res + s0 * a.ldr * b;
        cudaError_t e = cudaErrorInvalidValue;
        switch (a.tg->fmt) {
        case B200Q_I8: e = a.tu ? run<B200Q_I8, true>(c, st) : run<B200Q_I8, false>(c, st); break;
        case B200Q_I4: e = a.tu ? run<B200Q_I4, true>(c, st) : run<B200Q_I4, false>(c, st); break;
        case B200Q_I2: e = a.tu ? run<B200Q_I2, true>(c, st) : run<B200Q_I2, false>(c, st); break;
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t q8_take_error(unsigned int *code) {
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_q8_err, sizeof(unsigned int));
    if (e == cudaSuccess && *code) e = cudaMemcpyToSymbol(g_q8_err, &zero, sizeof(unsigned int));
    return e;
}

cudaError_t q8_selftest(long long wait_ns, unsigned int code) {
    const long long ns = wait_ns < 0 ? kWaitNs : wait_ns;
    cudaError_t e = cudaMemcpyToSymbol(g_q8_wait_ns, &ns, sizeof ns);
    if (e == cudaSuccess && code) e = cudaMemcpyToSymbol(g_q8_err, &code, sizeof code);
    return e;
}

}  // namespace qwq
