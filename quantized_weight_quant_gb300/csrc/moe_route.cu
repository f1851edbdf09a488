// The experts of each token: scores, grouped top-k and weights.
//     s = softmax(l) or 1 / (1 + e^-l),  c = s + bias  (no bias: c has the logits' order)
//     ids = the k largest c among the topk_group groups of the largest values,
//     w = s[ids] (/ their sum) * scale
// A warp per token: a lane holds every 32nd logit.  Bound: a call's latency for
// a few tokens, the issue of the k rounds of selection for many.
//   * Selection works on keys whose order as integers is that of the values, 0
//     for what cannot be chosen: a round is two integer reductions of the warp,
//     the largest key and the lowest index that has it.
//   * The order is that of the 64-bit formula.  f32 decides where the values that
//     a decision sets apart are further from each other than f32's errors;
//     otherwise the warp goes through the row once more in f64 (GB300 has few
//     f64 units: 256 sigmoids take longer than the rest of the row together).
//     Without a bias c has the logits' order, which is exact in f32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "launch.h"
#include "qwq_internal.h"

namespace qwq {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 4;                    // tokens per block where there are many

__device__ __forceinline__ float load(const float *p) { return *p; }
__device__ __forceinline__ float load(const __half *p) { return __half2float(*p); }
__device__ __forceinline__ float load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// What decides first: within 1e-6 of the scores is enough (keys_of's distances).
__device__ __forceinline__ float exp_of(float v) { return __expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }
__device__ __forceinline__ float ratio(float a, float b) { return __fdividef(a, b); }
__device__ __forceinline__ double ratio(double a, double b) { return a / b; }

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < INFINITY; }

// Integers in the order of the values; -infinity and NaN are 0, and -0 is 0.
__device__ __forceinline__ unsigned key_of(float v) {
    if (!(v > -INFINITY)) return 0u;
    const unsigned b = __float_as_uint(v + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ unsigned long long key_of(double v) {
    if (!(v > -INFINITY)) return 0ull;
    const unsigned long long b = (unsigned long long)__double_as_longlong(v + 0.0);
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ float value_of(unsigned k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ double value_of(unsigned long long k) {
    return __longlong_as_double((long long)(k >> 63 ? k & 0x7FFFFFFFFFFFFFFFull : ~k));
}

__device__ __forceinline__ unsigned warp_max(unsigned k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long k) {
    const unsigned hi = __reduce_max_sync(kAll, (unsigned)(k >> 32));
    const unsigned lo = __reduce_max_sync(kAll, (unsigned)(k >> 32) == hi ? (unsigned)k : 0u);
    return (unsigned long long)hi << 32 | lo;
}

template <class V> struct Key;
template <> struct Key<float> { using T = unsigned; };
template <> struct Key<double> { using T = unsigned long long; };

// e^(a - b): the difference's rounding, which grows with it, is made good.
__device__ __forceinline__ float exp_diff(float a, float b) {
    const float d = a - b, v = d - a;
    const float err = (a - (d - v)) - (b + v);         // exact (D. Knuth's two-sum)
    return err == err ? expf(d) * (1.f + err) : expf(d);
}

// One token's row: in this warp's registers, the logits in its shared memory too.
template <int NV> struct Row {
    float l[NV], bias[NV];                   // logit and bias of expert lane + 32 i, -infinity and 0 past E
    float *sm;                               // the same, by expert
    float top, sum;                          // softmax: the largest finite logit, sum exp(l - top) of those
    bool nan;
};

__device__ __forceinline__ unsigned first_lane(bool is) { return __ffs(__ballot_sync(kAll, is)) - 1; }

// The values of the groups, lane g that of group g, from c's keys, and the sums of the
// magnitudes in them, by which they are rounded (their signs may differ): of groups of
// 32 m neighbours the m registers' two largest over the warp; of 2, 4, 8 or 16 neighbours
// over as many lanes; of another number by a walk over c in shared memory.
template <int NV>
__device__ __forceinline__ float group_values(const Route &p, int lane, int n, const unsigned (&kc)[NV], float *by, float &size) {
    unsigned a = 0, b = 0;                   // of this lane's group: the two largest keys
    if (n % 32 == 0) {
        unsigned ga = 0, gb = 0;
        int g = 0, left = n / 32;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const unsigned x = __reduce_max_sync(kAll, kc[i]), at = first_lane(kc[i] == x);
            const unsigned y = p.group_top > 1 ? __reduce_max_sync(kAll, lane == (int)at ? 0u : kc[i]) : 0u;
            gb = max(min(ga, x), max(gb, y));
            ga = max(ga, x);
            if (--left == 0) {
                if (lane == g) a = ga, b = gb;
                ga = gb = 0;
                ++g;
                left = n / 32;
            }
        }
    } else if (n < 32 && (n & (n - 1)) == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unsigned x = kc[i], y = 0;
            for (int o = 1; o < n; o <<= 1) {
                const unsigned ox = __shfl_xor_sync(kAll, x, o), oy = __shfl_xor_sync(kAll, y, o);
                y = max(min(x, ox), max(y, oy));
                x = max(x, ox);
            }
            // group g is in register i = g n / 32, from lane g n % 32 on
            const int from = lane * n;
            const unsigned gx = __shfl_sync(kAll, x, from & 31), gy = __shfl_sync(kAll, y, from & 31);
            if (from >> 5 == i) a = gx, b = gy;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane + 32 * i < p.E) by[lane + 32 * i] = __uint_as_float(kc[i]);
        __syncwarp();
        if (lane < p.n_group) {
            int j = lane % n;                // lanes begin at different places: no bank conflicts
#pragma unroll 1
            for (int t = 0; t < n; ++t) {
                const unsigned v = __float_as_uint(by[lane * n + j]);
                b = max(min(a, v), b);
                a = max(a, v);
                if (++j == n) j = 0;
            }
        }
        __syncwarp();
    }
    size = 0.f;
    if (a == 0) return -INFINITY;
    const float va = value_of(a), vb = p.group_top > 1 && b ? value_of(b) : 0.f;
    size = fabsf(va) + fabsf(vb);
    return va + vb;
}
template <int NV>
__device__ __forceinline__ double group_values(const Route &p, int lane, int n, const unsigned long long (&kc)[NV], double *by, double &) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (lane + 32 * i < p.E) by[lane + 32 * i] = __longlong_as_double((long long)kc[i]);
    __syncwarp();
    unsigned long long a = 0, b = 0;
    if (lane < p.n_group) {
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
            const unsigned long long v = (unsigned long long)__double_as_longlong(by[lane * n + t]);
            b = max(min(a, v), b);
            a = max(a, v);
        }
    }
    __syncwarp();
    if (a == 0) return -INFINITY;
    return value_of(a) + (p.group_top > 1 && b ? value_of(b) : 0.);
}

// Keys of c in the arithmetic of V; the groups that do not stay have key 0.
// *near: a decision was nearer than V's errors (f32 only).
template <class V, int NV>
__device__ __forceinline__ void keys_of(const Route &p, const Row<NV> &r, int lane, typename Key<V>::T (&key)[NV],
                                        bool *near) {
    V sum = (V)r.sum;
    if (sizeof(V) == 8 && p.score == B200Q_SCORE_SOFTMAX) {
        sum = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) sum += finite(r.l[i]) ? exp_of((V)r.l[i] - (V)r.top) : (V)0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    }
    // c, or where nothing but its order counts, the logit
    const bool scored = p.bias || (p.n_group > 1 && p.group_top > 1);
    typename Key<V>::T kc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const float l = r.l[i];
        V c = (V)l;
        if (scored) {
            if (p.score == B200Q_SCORE_SOFTMAX) c = finite(l) ? ratio(exp_of((V)l - (V)r.top), sum) : (V)0;
            else c = ratio((V)1, (V)1 + exp_of(-(V)l));
            c += (V)r.bias[i];
        }
        kc[i] = l > -INFINITY ? key_of(c) : (typename Key<V>::T)0;
        key[i] = p.bias ? kc[i] : key_of((V)l);
    }
    if (p.n_group == 1) return;
    const int n = p.E / p.n_group;
    V size = 0;
    const V value = group_values<NV>(p, lane, n, kc, reinterpret_cast<V *>(r.sm + p.E + (p.E & 1)), size);
    // place: how many groups have a larger value, or the same and a lower index
    int place = 0;
    V least = INFINITY;                      // to the next lower or equal value
#pragma unroll 1
    for (int g = 0; g < p.n_group; ++g) {
        const V o = __shfl_sync(kAll, value, g);
        if (o > value || (o == value && g < lane)) ++place;
        else if (g != lane) least = value - o < least ? value - o : least;
    }
    const unsigned stays = __ballot_sync(kAll, lane < p.n_group && place < p.topk_group);
    if (near && scored && p.topk_group < p.n_group) {
        // Only the last group that stays has to be told from the next.  Sums that are infinite or NaN are left to f64.
        const bool last = lane < p.n_group && place == p.topk_group - 1 && value > -INFINITY;
        const float most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint((float)size)));
        const float eps = (p.score == B200Q_SCORE_SOFTMAX ? 1.2e-5f : 1.8e-6f) + 3e-7f * most;
        if (__any_sync(kAll, (last && !((float)least > eps)) || !(most < INFINITY))) *near = true;
    }
    const Quotient &by_n = p.by_group;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        if (e < p.E && !(stays >> by_n(e) & 1u)) key[i] = 0;
    }
}

// The k largest keys, descending, equal ones by index: lane j gets the j-th
// expert, or -1.  near: as above, of neighbouring choices, the last and the one after
// it (lane k's) among them; *least is then the least value of those.
template <class V, int NV>
__device__ __forceinline__ int select(const Route &p, int lane, typename Key<V>::T (&key)[NV], bool *near, float *least) {
    using K = typename Key<V>::T;
    int mine = -1;
    const float eps = p.score == B200Q_SCORE_SOFTMAX ? 6e-6f : 9e-7f;
    float before = INFINITY;
    const int rounds = near && p.bias ? p.k + 1 : p.k;
#pragma unroll 1
    for (int j = 0; j < rounds; ++j) {
        K best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i] > best) best = key[i], at = i;        // ascending i: the lowest index of equal ones
        const K top = warp_max(best);
        if (top == 0) break;
        const unsigned e = __reduce_min_sync(kAll, best == top ? (unsigned)(lane + 32 * at) : kAll);
        if (near && p.bias) {
            const float v = (float)value_of(top);
            if (j > 0 && !(before - v > eps + 1.5e-7f * fabsf(v))) *near = true;
            before = v;
        }
        if (lane == j) mine = (int)e;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((unsigned)(lane + 32 * i) == e) key[i] = 0;
    }
    if (least) *least = before;
    return mine;
}

// Where f32 left the order of neighbouring choices open: those that it looked at
// (id), and what is no further below the last of them than its errors, are ranked
// in 64 bits, a lane each.  key: what is left of the row's, f32.  false: more than
// 32 of them, or a softmax, which needs the whole row.
template <int NV>
__device__ __forceinline__ bool rank_again(const Route &p, const Row<NV> &r, int lane, const unsigned (&key)[NV], float least, int &id) {
    const float floor_ = least - 9e-7f - 1.5e-7f * fabsf(least);
    if (!finite(floor_) || p.score == B200Q_SCORE_SOFTMAX || p.k == 32) return false;
    int have = __popc(__ballot_sync(kAll, id >= 0)), mine = id;
    const unsigned low = key_of(floor_);
#pragma unroll 1
    for (int i = 0; i < NV; ++i) {
        unsigned k = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j == i) k = key[j];
        unsigned in = __ballot_sync(kAll, k != 0 && k >= low);
        if (have + __popc(in) > 32) return false;
#pragma unroll 1
        for (; in; in &= in - 1, ++have)
            if (lane == have) mine = 32 * i + __ffs(in) - 1;
    }
    unsigned long long k64 = 0;
    if (lane < have) k64 = key_of(1.0 / (1.0 + exp(-(double)r.sm[mine])) + (double)p.bias[mine]);
    int got = -1;
#pragma unroll 1
    for (int j = 0; j < p.k; ++j) {
        const unsigned long long top = warp_max(k64);
        if (top == 0) break;
        const unsigned e = __reduce_min_sync(kAll, k64 == top ? (unsigned)mine : kAll);
        if (lane == j) got = (int)e;
        if (k64 == top && mine == (int)e) k64 = 0;
    }
    id = got;
    return true;
}

template <class T, int NV>
__global__ void __launch_bounds__(32 * kWarps) moe_route_kernel(const Route p, int row_bytes) {
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long s = (long long)blockIdx.x * (blockDim.x >> 5) + warp;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (s >= p.S) return;                    // whole warps; no block barrier below
    const T *src = (const T *)p.logits + s * p.ld;
    Row<NV> r;
    r.sm = reinterpret_cast<float *>(smem + warp * row_bytes);
    r.nan = false;
    r.top = -INFINITY;
    r.sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) r.l[i] = lane + 32 * i < p.E ? load(src + lane + 32 * i) : -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) r.bias[i] = p.bias && lane + 32 * i < p.E ? p.bias[lane + 32 * i] : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        if (e < p.E) {
            r.sm[e] = r.l[i];
            r.nan |= r.l[i] != r.l[i] || r.bias[i] != r.bias[i];
        }
        if (finite(r.l[i])) r.top = fmaxf(r.top, r.l[i]);
        else r.nan |= p.score == B200Q_SCORE_SOFTMAX && r.l[i] > 0.f;      // infinity / infinity
    }
    r.nan = __any_sync(kAll, r.nan);
    if (p.score == B200Q_SCORE_SOFTMAX) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) r.top = fmaxf(r.top, __shfl_xor_sync(kAll, r.top, o));
#pragma unroll
        for (int i = 0; i < NV; ++i) r.sum += finite(r.l[i]) ? __expf(r.l[i] - r.top) : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) r.sum += __shfl_xor_sync(kAll, r.sum, o);
    }
    bool near = false, near_groups = false;
    unsigned key[NV];
    float least;
    __syncwarp();                            // the logits in shared memory
    keys_of<float>(p, r, lane, key, &near_groups);
    int id = select<float>(p, lane, key, &near, &least);
    if (near_groups || (near && !rank_again(p, r, lane, key, least, id))) {
        unsigned long long k64[NV];
        keys_of<double>(p, r, lane, k64, nullptr);
        id = select<double>(p, lane, k64, nullptr, nullptr);
    }
    if (lane >= p.k) id = -1;
    __syncwarp();
    // weights: lane j its own.  With norm only the ratios count: they are taken
    // relative to the largest logit chosen (capped at 0 for the sigmoid), so that
    // scores too small for f32 still have their ratios.
    const bool have = id >= 0;
    const float l = have ? r.sm[id] : -INFINITY;
    float w, most = l;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, o));
    if (p.score == B200Q_SCORE_SOFTMAX) {
        w = p.norm ? exp_diff(l, most) : exp_diff(l, r.top) / r.sum;
    } else if (l > 0.f || !p.norm) {
        w = 1.f / (1.f + expf(-l));
    } else {
        w = exp_diff(l, fminf(most, 0.f)) / (1.f + expf(l));
    }
    if (!have) w = 0.f;
    if (p.norm) {
        float sum = w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (have) w /= sum;
    }
    w *= p.scale;
    if (r.nan) w = __int_as_float(0x7FC00000);
    if (lane < p.k) {
        p.ids[s * p.k + lane] = id;
        p.wts[s * p.k + lane] = w;
    }
}

template <class T, int NV>
cudaError_t start(const Route &a, cudaStream_t st) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int warps = a.S > 2 * sm_count(dev) ? kWarps : 1;
    // a row's logits, and where there are groups their c as f64
    Route p = a;
    p.by_group = Quotient(a.E / a.n_group);
    const int row_bytes = ((a.E + (a.E & 1)) * 4 + (a.n_group > 1 ? a.E * 8 : 0) + 15) & ~15;
    return launch_dependent(moe_route_kernel<T, NV>, dim3((unsigned)((a.S + (long long)warps - 1) / warps)), 32 * warps,
                            (size_t)warps * row_bytes, st, p, row_bytes);          // at most 4 * 12 KB
}

template <class T>
cudaError_t run(const Route &a, cudaStream_t st) {
    if (a.E <= 32) return start<T, 1>(a, st);
    if (a.E <= 64) return start<T, 2>(a, st);
    if (a.E <= 128) return start<T, 4>(a, st);
    if (a.E <= 256) return start<T, 8>(a, st);
    if (a.E <= 512) return start<T, 16>(a, st);
    return start<T, 32>(a, st);
}

}  // namespace

cudaError_t launch_moe_route(const Route &a, cudaStream_t st) {
    switch (a.type) {
    case B200Q_T_F32: return run<float>(a, st);
    case B200Q_T_F16: return run<__half>(a, st);
    default: return run<__nv_bfloat16>(a, st);
    }
}

}  // namespace qwq
