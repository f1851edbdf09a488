// The experts' layer for a few tokens, routed on the device.
//     h[s,j] = act(gate_e x[s]) * (up_e x[s]),   y[s] = res[s] + sum_j wts[s,j] down_e h[s,j],   e = ids[s,j]
//
// Bound: HBM, the three matrices of every expert that some token has, each read
// once.  A slot (s, j) is a column of its expert's products.
//   * Each block makes the plan from the ids itself: the slots in the order of
//     their experts, cut into chunks of nc columns.  The work is chunks x
//     slices of the rows' length x tiles of 16 rows, in that order, and a block
//     takes an even run of tiles, so that it holds the columns of one or two
//     experts in its lifetime.
//   * A tile is 16 rows for the warp-level tensor instruction m16n8k16: 16 rows
//     of down, or 8 of gate and the same 8 of up, whose sums then meet in one
//     thread.  A column is scaled by a power of two into f16's range, in two
//     pieces where its type needs them (moe_pieces).  Sums are f32, taken out of the
//     tensor instruction's accumulator, which truncates, every 128 bytes of a row
//     (1024 where there are many columns, every 4 where there are two pieces).
//   * Codes are signed, exact in f16: one AND and one packed f16 FMA for two of them.
//     A code of 0 then adds nothing, whatever it meets.  (Unsigned ones, the zero
//     point times the column's sum taken off at the end, save the FMA, 5 to 10 % of a
//     call; but their error goes by the column's largest value instead of by sum |deq x|:
//     a value 10^3 times the rest on a weight of 0 left errors 1 to 11 times the stated ones.)
//   * Few columns (moe_few_kernel, up to 8 per expert): the columns stay in shared
//     memory.  A warp has its own ring of codes, brought by its own TMA boxes of 8
//     rows x 128 bytes several lines ahead and across the tiles of the run: no
//     barrier of the block orders them.  A warp takes whole tiles where the block has many;
//     otherwise wk warps take the 128-byte lines of a tile in turn and add their
//     sums in warp order.  Three launches: gate and up, down, the weighted sum; from
//     three tokens on their rows are prepared by one before.
//   * Many columns (moe_many_kernel), where there are tiles for all SMs: the rows are prepared once, in a launch before
//     each product, and come line by line beside the codes.
// No sum depends on the order in which blocks run.
#include <atomic>

#include "moe.h"
#include "qmat_q8.h"

namespace qwq {
namespace {

__device__ unsigned int g_moe_err = 0;        // first error a kernel recorded (a B200Q_E* code, negated)
constexpr long long kMoeWaitNs = 2000000000;
std::atomic<long long> g_moe_wait_ns{kMoeWaitNs};   // b200q_selftest_moe shortens it
std::atomic<int> g_moe_withheld{0};

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
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long s = blockIdx.y;
    const int o = blockIdx.x * 128 + threadIdx.x;
    if (o >= p.D) return;
    float y = 0.f;
    for (int j0 = 0; j0 < p.k; j0 += 8) {      // eight slots' loads at a time
        float v[8], w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const long long at = s * p.k + j0 + j;
            const int e = j0 + j < p.k ? p.ids[at] : -1;
            const bool have = e >= 0 && e < p.E;
            w[j] = have ? p.wts[at] : 0.f;
            v[j] = have ? p.part[at * p.D + o] : 0.f;
            for (int n = 1; n < p.ns; ++n) v[j] += have ? p.part[((long long)n * p.P + at) * p.D + o] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) y = fmaf(w[j], v[j], y);
    }
    if (p.res) y += load_typed(p.res, s * p.ldr + o, p.type);
    store_typed(p.y, s * p.ldy + o, p.type, y);
}

// ---------------------------------------------------------------- launches
// Which kernel takes the products: the columns that an expert has on average and
// twice their root more.
int kind_of(int S, int k, int E) {
    const double avg = (double)S * k / E;
    double root = 1.0;
    while (root * root < avg) root += 0.5;
    if (S <= 2) return 1;
    return S <= 8 || avg + 2.0 * root <= 8.0 ? 0 : 2;
}

// log2 of the warps that share a tile, of blocks with t tiles of `per` lines each:
// the largest share of the warps' lines that is used, in rounds of warps / 2^wk
// tiles; sharing costs a barrier and an addition per tile.
int shared_by(int warps, double t, int per) {
    int best = 0;
    double most = 0.;
    for (int wk = 0; 1 << wk <= warps && 1 << wk <= per; ++wk) {
        const int g = warps >> wk, w = 1 << wk;
        const double rounds = (double)((long long)(t / g + 0.999)), lines = (per + w - 1) / w * w;
        const double used = t / ((rounds < 1. ? 1. : rounds) * g) * per / lines * (1. - (wk ? 0.02 * w : 0.));
        if (used > most) most = used, best = wk;
    }
    return best;
}

// Experts that S tokens with k slots each are expected to have chosen among E.
double chosen(int S, int k, int E) {
    double none = 1.;
    for (int s = 0; s < S; ++s) none *= k < E ? 1. - (double)k / E : 0.;
    return E * (1. - none);
}

// Steps of a warp, a line of a tile each, that the two kernels need for a product.
// Many columns: a block takes 16 tiles together, so that a few tiles leave SMs
// idle however long their rows are; few columns: warps take tiles, or share them.
struct Steps {
    double few, many;
};
Steps steps_of(int S, int k, int E, int tiles, int lines, int nc, int n_sms) {
    const double touched = chosen(S, k, E), avg = S * (double)k / touched;
    const double chunks8 = touched * (avg / kMoeFewColumns + 0.5), chunks = touched * (avg <= 0.75 * nc ? 1. : avg / nc + 0.5);
    const double rounds = chunks * ((tiles + 15) / 16);
    return {chunks8 * tiles * lines / (16. * n_sms), (double)((long long)(rounds / n_sms + 0.999)) * lines};
}

template <int FMT>
cudaError_t run(const Moe &a, cudaStream_t st) {
    constexpr int KC = FMT == B200Q_I8 ? 16 : FMT == B200Q_I4 ? 32 : 64;
    const Experts &ex = *a.ex;
    const int b = a.type == B200Q_T_F32 ? 4 : 2;
    int part = kMoePairs / a.k < kMoeTokens ? kMoePairs / a.k : kMoeTokens;            // tokens per launch
    const int in_lines = (int)(ex.ld_in / 128), out_lines = (int)(ex.ld_out / 128);
    const int pc_in = moe_pieces(a.type, false), pc_out = moe_pieces(a.type, true);
    const int n_sms = sm_count(ex.device);
    int S = 0, P = 0, kind = 0;
    MoeWay wi, wo;
    for (;; part /= 2) {
        S = a.S < part ? a.S : part, P = S * a.k, kind = kind_of(S, a.k, ex.E);
        wi = moe_way<FMT>(kind, pc_in, S, in_lines), wo = moe_way<FMT>(kind, pc_out, S, out_lines);
        if (kind == 2) {
            // What staging costs the kernel for few columns is about three steps; two pieces cost the other a quarter more.
            // Few and many columns, us (steps): int8 6144 / 256, 8 experts, f32, 64 tokens of 2: 52 and 102 (19 and 52); int8
            // 2048 / 1024, 4 experts, f32, 64 of 2: 46 and 59 (23 and 24); int8 1024 / 2048, 4 experts, f16, 48 of 2: 39 and
            // 51; int4 2048 / 1024, 32 experts, bf16, 64 of 4: 60 and 52 (30 and 24); int4 1024 / 512, 16 experts, bf16, 32
            // of 4: 23 and 21 (4 and 6); int4 4096 / 4096, 8 experts, bf16, 64 of 2: 135 and 93; int2 2048 / 2048, 8
            // experts, bf16, 40 of 4: 48 and 36.
            const Steps i = steps_of(S, a.k, ex.E, (int)((ex.F + 7ll) / 8), in_lines, wi.nc, n_sms);
            const Steps o = steps_of(S, a.k, ex.E, (int)((ex.D + 15ll) / 16), out_lines, wo.nc, n_sms);
            if (i.few + o.few + 3. < (pc_in == 2 ? 1.25 : 1.) * i.many + (pc_out == 2 ? 1.25 : 1.) * o.many) {
                kind = 0;
                wi = moe_way<FMT>(kind, pc_in, S, in_lines), wo = moe_way<FMT>(kind, pc_out, S, out_lines);
            }
        }
        if (kind == 1 && (wi.ns > 1 || wo.ns > 1)) {       // two blocks on an SM are not worth slices
            kind = 0;
            wi = moe_way<FMT>(kind, pc_in, S, in_lines), wo = moe_way<FMT>(kind, pc_out, S, out_lines);
        }
        // tiles of all chunks are numbered in 31 bits; at kMoeMaxSize rows and columns one token's are
        if (part == 1 || ((long long)P * wi.ns * (ex.F / 8 + 1) < 1 << 30 && (long long)P * wo.ns * (ex.D / 16 + 1) < 1 << 30)) break;
    }
    auto place = [&](MoeStream &p, const MoeWay &w, int n) {
        p.by_tiles = Quotient(p.tiles);
        p.by_grid = Quotient(n_sms * w.blocks);
        p.by_k = Quotient(a.k);
        p.by_rounds = Quotient((p.tiles + 15) / 16);
        p.wk = shared_by(w.warps, chosen(n, a.k, ex.E) * w.ns * p.tiles / (n_sms * w.blocks), p.lines / w.ns);
        p.ns = w.ns;
        p.nc = w.nc;
        p.held = w.held;
        p.pitch = w.pitch;
    };
    const int ldh = (ex.F + 7) / 8 * 8;
    // h, the down sums, and for many columns the prepared rows
    auto up16 = [](size_t n) { return (n + 15) / 16 * 16; };
    const size_t n_h = up16((size_t)wi.ns * P * (wi.ns == 1 ? 1 : 2) * ldh * 4), n_part = up16((size_t)wo.ns * P * ex.D * 4);
    // Tokens' rows are prepared by a launch of their own where there are more than
    // two (every block would convert them all), h where there are many columns.
    const bool prepare = kind != 1 && S > 2;
    const size_t n_x = kind == 2 ? (size_t)P * pc_in * in_lines * (16 * KC + 64) : prepare ? (size_t)S * pc_in * in_lines * 16 * KC : 0;
    const size_t n_hc = kind == 2 ? (size_t)P * pc_out * out_lines * (16 * KC + 64) : 0;
    const size_t n_info = prepare ? up16((size_t)P * 4) : 0;
    uint8_t *ws = nullptr;
    cudaError_t e = workspace_alloc((void **)&ws, n_h + n_part + (n_x > n_hc ? n_x : n_hc) + n_info, st);
    if (e != cudaSuccess) return e;
    float *h = (float *)ws, *sums = (float *)(ws + n_h);
    float *info = (float *)(ws + n_h + n_part);
    uint8_t *cols = ws + n_h + n_part + n_info;
    for (int s0 = 0; s0 < a.S && e == cudaSuccess; s0 += part) {
        const int n = a.S - s0 < part ? a.S - s0 : part;
        MoeStream p{};
        p.table = ex.table;
        p.ids = a.ids + (long long)s0 * a.k;
        p.x = (const char *)a.x + s0 * a.ldx * b;
        p.in = h;
        p.out = h;
        p.err = ex.err;
        p.ldx = a.ldx;
        p.S = n;
        p.P = n * a.k;
        p.k = a.k;
        p.E = ex.E;
        p.type = a.type;
        p.act = a.act;
        p.K = ex.D;
        p.rows = ex.F;
        p.ldh = ldh;
        p.aligned = (uintptr_t)p.x % 16 == 0 && a.ldx * b % 16 == 0;
        p.lines = in_lines;
        p.ns_in = wi.ns;
        p.tiles = (int)((ex.F + 7ll) / 8);
        place(p, wi, n);
        p.cols = cols;
        p.info = info;
        p.prepared = prepare;
        p.wait_ns = (unsigned long long)g_moe_wait_ns.load(std::memory_order_relaxed);
        p.withheld = g_moe_withheld.load(std::memory_order_relaxed);
        if (prepare) e = moe_launch_prepare<FMT>(p, n, kind == 2, cols, info, st);
        if (e == cudaSuccess) e = moe_launch_stream<FMT>(p, wi, n_sms, st);
        if (e != cudaSuccess) break;
        p.down = true;
        p.out = sums;
        p.K = ex.F;
        p.rows = ex.D;
        p.lines = out_lines;
        p.tiles = (int)((ex.D + 15ll) / 16);
        place(p, wo, n);
        p.prepared = kind == 2;
        if (p.prepared) e = moe_launch_prepare<FMT>(p, p.P, true, cols, info, st);
        if (e == cudaSuccess) e = moe_launch_stream<FMT>(p, wo, n_sms, st);
        if (e != cudaSuccess) break;
        Sum q{sums, p.ids, a.wts + (long long)s0 * a.k, a.res ? (const char *)a.res + s0 * a.ldr * b : nullptr,
              (char *)a.y + s0 * a.ldy * b, a.ldr, a.ldy, p.P, a.k, ex.E, ex.D, wo.ns, a.type};
        e = launch_dependent(moe_sum_kernel, dim3((unsigned)((ex.D + 127ll) / 128), n), 128, 0, st, q);
    }
    cudaError_t e2 = workspace_free(ws, st);
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

// What a call could not do while its stream is captured, done when the handle is
// made: the lookup of the error word, which may load device code, and the
// making of the workspaces' pool.
cudaError_t moe_make_ready(unsigned int **err, cudaStream_t st) {
    void *ws = nullptr;
    cudaError_t e = cudaGetSymbolAddress((void **)err, g_moe_err);
    if (e == cudaSuccess) e = workspace_alloc(&ws, 16, st);
    if (e == cudaSuccess) e = workspace_free(ws, st);
    return e;
}

void moe_selftest(long long wait_ns, bool withhold) {
    g_moe_wait_ns.store(wait_ns < 0 ? kMoeWaitNs : wait_ns, std::memory_order_relaxed);
    g_moe_withheld.store(withhold ? 16 : 0, std::memory_order_relaxed);
}

// Reads and clears the error word (0: none).
cudaError_t moe_take_error(unsigned int *code) {
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_moe_err, sizeof(unsigned int));
    if (e == cudaSuccess && *code) e = cudaMemcpyToSymbol(g_moe_err, &zero, sizeof(unsigned int));
    return e;
}

}  // namespace qwq
