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

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

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

// One token's row: the logits in this warp's registers and its shared memory.
template <int NV> struct Row {
    float l[NV];                             // logit of expert lane + 32 i, -infinity past E
    float *sm;                               // the same, by expert
    float top, sum;                          // softmax: the largest finite logit, sum exp(l - top) of those
    bool nan;
};

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
    auto score = [&](float l) {
        if (p.score == B200Q_SCORE_SOFTMAX) return finite(l) ? exp_of((V)l - (V)r.top) / sum : (V)0;
        return (V)1 / ((V)1 + exp_of(-(V)l));
    };
    // c, or where nothing but its order counts, the logit
    const bool scored = p.bias || (p.n_group > 1 && p.group_top > 1);
    V c[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        c[i] = (V)r.l[i];
        if (r.l[i] != r.l[i]) c[i] = -INFINITY;
        if (scored && c[i] > -INFINITY) {
            c[i] = score(r.l[i]);
            if (p.bias) c[i] += (V)p.bias[e];
        }
        key[i] = key_of(c[i]);
        if (!p.bias) key[i] = (typename Key<V>::T)(e < p.E ? key_of((V)(r.l[i])) : key_of((V)-INFINITY));
    }
    if (p.n_group == 1) return;
    // a lane per group; c by expert, in the arithmetic of V
    V *by = reinterpret_cast<V *>(r.sm + p.E + (p.E & 1));
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (lane + 32 * i < p.E) by[lane + 32 * i] = key_of(c[i]) ? c[i] : (V)-INFINITY;
    __syncwarp();
    const int n = p.E / p.n_group;
    V a = -INFINITY, b = -INFINITY;          // the group's two largest
    if (lane < p.n_group) {
        int j = lane % n;                    // lanes begin at different places: no bank conflicts
        for (int t = 0; t < n; ++t) {
            const V v = by[lane * n + j];
            b = v > a ? a : v > b ? v : b;
            a = v > a ? v : a;
            if (++j == n) j = 0;
        }
    }
    V value = a;
    if (p.group_top > 1 && b > -INFINITY) value += b;
    __syncwarp();
    // place: how many groups have a larger value, or the same and a lower index
    int place = 0;
    V least = INFINITY;                      // to the next lower or equal value
    for (int g = 0; g < p.n_group; ++g) {
        const V o = __shfl_sync(kAll, value, g);
        if (o > value || (o == value && g < lane)) ++place;
        else if (g != lane) least = value - o < least ? value - o : least;
    }
    const unsigned stays = __ballot_sync(kAll, lane < p.n_group && place < p.topk_group);
    if (near && scored) {
        // only the last group that stays has to be told from the next.  A value that is infinite or NaN is left to f64.
        const bool last = lane < p.n_group && place == p.topk_group - 1 && p.topk_group < p.n_group && value > -INFINITY;
        const float eps = (p.score == B200Q_SCORE_SOFTMAX ? 1.2e-5f : 4e-6f) + 5e-7f * fabsf((float)value);
        if (__any_sync(kAll, last && !((float)least > eps))) *near = true;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        if (e < p.E && !(stays >> (e / n) & 1u)) key[i] = 0;
    }
}

// The k largest keys, descending, equal ones by index: lane j gets the j-th
// expert, or -1.  near: as above, of neighbouring choices.
template <class V, int NV>
__device__ __forceinline__ int select(const Route &p, int lane, typename Key<V>::T (&key)[NV], bool *near) {
    using K = typename Key<V>::T;
    int mine = -1;
    const float eps = p.score == B200Q_SCORE_SOFTMAX ? 6e-6f : 2e-6f;
    float before = INFINITY;
    const int rounds = near && p.bias ? p.k + 1 : p.k;       // one more: what the last choice was told from
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
            if (j > 0 && !(before - v > eps + 2.5e-7f * fabsf(v))) *near = true;
            before = v;
        }
        if (j < p.k && lane == j) mine = (int)e;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((unsigned)(lane + 32 * i) == e) key[i] = 0;
    }
    return mine;
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
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        if (e < p.E) {
            r.sm[e] = r.l[i];
            r.nan |= r.l[i] != r.l[i] || (p.bias && p.bias[e] != p.bias[e]);
        }
        if (finite(r.l[i])) r.top = fmaxf(r.top, r.l[i]);
        else r.nan |= p.score == B200Q_SCORE_SOFTMAX && r.l[i] > 0.f;      // infinity / infinity
    }
    r.nan = __any_sync(kAll, r.nan);
    if (p.score == B200Q_SCORE_SOFTMAX) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) r.top = fmaxf(r.top, __shfl_xor_sync(kAll, r.top, o));
#pragma unroll
        for (int i = 0; i < NV; ++i) r.sum += finite(r.l[i]) ? expf(r.l[i] - r.top) : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) r.sum += __shfl_xor_sync(kAll, r.sum, o);
    }
    bool near = false;
    unsigned key[NV];
    keys_of<float>(p, r, lane, key, &near);
    int id = select<float>(p, lane, key, &near);
    if (near) {
        unsigned long long k64[NV];
        keys_of<double>(p, r, lane, k64, nullptr);
        id = select<double>(p, lane, k64, nullptr);
    }
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
    const int row_bytes = ((a.E + (a.E & 1)) * 4 + (a.n_group > 1 ? a.E * 8 : 0) + 15) & ~15;
    return launch_dependent(moe_route_kernel<T, NV>, dim3((unsigned)((a.S + (long long)warps - 1) / warps)), 32 * warps,
                            (size_t)warps * row_bytes, st, a, row_bytes);          // at most 4 * 12 KB
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
