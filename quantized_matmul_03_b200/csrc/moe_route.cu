// moe_route.cu -- routing to experts: per token the top_k experts by score,
// and their weights.
//
// Mathematics.  s = softmax(l) or sigmoid(l) over the E logits of a token.  The
// experts are ordered by key = l (without a bias: both score functions grow
// with l) or s + bias; with groups, only the experts of the best topk_groups
// groups are candidates, a group's score being the sum of its group_top best
// s + bias (s without a bias).  Equal keys go to the lower index.  Weights are
// the chosen s, divided by their sum if renormalize, times scale.
//
// One warp per token, lane l holding experts l, l + 32, ...; each of the top_k
// rounds is a warp maximum and a warp minimum of the indices that reach it
// (two redux instructions), after which only the owner looks for its next
// best.  The kernel reads the logits once and writes 8 bytes per slot; small
// batches are bound by the launch, long ones by the rounds' latency.
//
// Exactness of the choice.  Keys s + bias computed in fp32 carry an error that
// could exchange two experts whose keys nearly coincide.  The fp32 pass
// therefore bounds its error and checks the gap between every pair of
// neighbours in the order it found (the last chosen and the best rejected one
// too, for experts and for groups); a token with a gap inside the bound is
// ordered again with fp64 keys.  Logits as keys need no such check.
#include <type_traits>

#include "moe.cuh"
#include "ptx_sm100.cuh"

namespace qmm {
namespace {

constexpr int kRouteWarps = 4;  // tokens per CTA

struct RouteParams {
    const void *logits;
    const float *bias;
    int32_t *indices;
    float *weights;
    int64_t T;
    int E, k, n_groups, topk_groups, group_top, gsize;
    int renormalize;
    double scale;
};

// Order-preserving integer keys: greater float, greater key.  NaN is 1, below
// every number; 0 is left for "not a candidate".  -0 counts as +0.
__device__ __forceinline__ uint32_t key_of(float v) {
    if (v != v) return 1u;
    const uint32_t b = __float_as_uint(v + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ uint64_t key_of(double v) {
    if (v != v) return 1ull;
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return ((uint64_t)hi << 32) | lo;
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The k best of key[V] (lane l: experts l + 32 i); lane j returns the j-th
// one's index.  Keys are consumed.  check(j, key) sees the j-th best key, for
// `rounds` >= k rounds (key 0: no candidate is left).
template <int V, typename Key, typename Check>
__device__ __forceinline__ int select_top(Key (&key)[V], int k, int rounds, int lane, Check check) {
    Key best = 0;
    int bi = 0;
    auto rescan = [&]() {
        best = key[0];
        bi = 0;
#pragma unroll
        for (int i = 1; i < V; ++i)
            if (key[i] > best) {
                best = key[i];
                bi = i;
            }
    };
    rescan();
    int mine = 0;
    for (int j = 0; j < rounds; ++j) {
        const Key mx = warp_max(best);
        const uint32_t at = __reduce_min_sync(0xffffffffu, best == mx ? (uint32_t)(bi * 32 + lane) : 0xffffffffu);
        if (j < k && lane == j) mine = (int)at;
        check(j, mx);
        if ((at & 31u) == (uint32_t)lane) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == bi) key[i] = 0;
            rescan();
        }
    }
    return mine;
}

template <int V, typename F, int SCORE>
__device__ __forceinline__ void scores_of(const float (&l)[V], int lane, int E, F (&s)[V]) {
    if constexpr (SCORE == QMM_SCORE_SIGMOID) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (std::is_same<F, double>::value) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
            else s[i] = 1.f / (1.f + expf(-l[i]));
        }
    } else {
        float m = __uint_as_float(0xff800000u);
#pragma unroll
        for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);  // (fmaxf passes over NaN)
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        F z = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            // The largest logit's term is 1 also where it is infinite; a token
            // whose logits are all -inf has no terms.
            if (m == __uint_as_float(0xff800000u)) s[i] = 0;
            else if (l[i] == m) s[i] = 1;
            else if constexpr (std::is_same<F, double>::value) s[i] = exp((double)l[i] - (double)m);
            else s[i] = expf(l[i] - m);
            if (lane + 32 * i < E) z += s[i];
        }
        z = warp_sum(z);
        const F inv = z > 0 ? F(1) / z : z;  // NaN stays NaN
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = std::is_same<F, double>::value ? (z > 0 ? s[i] / z : z) : s[i] * inv;
    }
}

// Candidates of the best groups: clears the keys of every other group.  sel:
// the values groups are scored by.  Returns false if the last group kept and
// the best one left out lie within tol of each other.
template <int V, typename Key, typename F>
__device__ __forceinline__ bool keep_groups(Key (&key)[V], const F (&sel)[V], const RouteParams &p, int lane,
                                            F tol) {
    const int G = p.n_groups;
    Key mine = 0;  // lane g: group g's score as a key
    F mine_v = 0;
    for (int g = 0; g < G; ++g) {
        Key b1 = 0, b2 = 0;
        F v1 = 0, v2 = 0;
        bool h2 = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            if (e >= g * p.gsize && e < (g + 1) * p.gsize) {
                const Key q = key_of(sel[i]);
                if (q > b1) {
                    b2 = b1; v2 = v1; h2 = b1 != 0;
                    b1 = q; v1 = sel[i];
                } else if (q > b2) {
                    b2 = q; v2 = sel[i]; h2 = true;
                }
            }
        }
        const Key m1 = warp_max(b1);
        const int o1 = __ffs(__ballot_sync(0xffffffffu, b1 == m1)) - 1;
        F sum = __shfl_sync(0xffffffffu, v1, o1);
        if (p.group_top == 2 && p.gsize > 1) {
            const bool own = lane == o1;
            const Key c = own ? (h2 ? b2 : Key(0)) : b1;
            const F cv = own ? v2 : v1;
            const Key m2 = warp_max(c);
            const int o2 = __ffs(__ballot_sync(0xffffffffu, c == m2)) - 1;
            sum += __shfl_sync(0xffffffffu, cv, o2);
        }
        if (lane == g) {
            mine = key_of(sum);
            mine_v = sum;
        }
    }
    unsigned live = 0;
    bool sure = true;
    F last = 0;
    for (int j = 0; j <= p.topk_groups && j < G; ++j) {
        const Key mx = warp_max(mine);
        const int g = __ffs(__ballot_sync(0xffffffffu, mine == mx)) - 1;
        const F v = __shfl_sync(0xffffffffu, mine_v, g);
        if (j < p.topk_groups) {
            live |= 1u << g;
            last = v;
        } else if (last - v <= tol) {
            sure = false;
        }
        if (lane == g) mine = 0;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        if (e < p.E && !((live >> (e / p.gsize)) & 1u)) key[i] = 0;
    }
    return sure;
}

// The token's order from fp64 scores.
template <typename T, int V, int SCORE>
__device__ __noinline__ int route_fp64(const T *row, const RouteParams &p, int lane) {
    float l[V];
    double s[V];
    uint64_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < p.E ? Dt<T>::to_f(row[e]) : __uint_as_float(0xff800000u);
    }
    scores_of<V, double, SCORE>(l, lane, p.E, s);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        if (p.bias && e < p.E) s[i] += (double)__ldg(p.bias + e);
        key[i] = e < p.E ? (p.bias ? key_of(s[i]) : key_of((double)l[i])) : 0ull;
    }
    if (p.n_groups > 1) keep_groups<V, uint64_t, double>(key, s, p, lane, -1.0);
    return select_top<V, uint64_t>(key, p.k, p.k, lane, [](int, uint64_t) {});
}

template <typename T, int V, int SCORE>
__global__ void __launch_bounds__(32 * kRouteWarps) moe_route_kernel(const RouteParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const T *row = static_cast<const T *>(p.logits) + t * p.E;
    float l[V];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < p.E ? Dt<T>::to_f(row[e]) : __uint_as_float(0xff800000u);
        nan = nan || l[i] != l[i];
    }
    nan = __any_sync(0xffffffffu, nan);

    uint32_t key[V];
    float s[V];
    if (p.bias != nullptr || p.n_groups > 1) scores_of<V, float, SCORE>(l, lane, p.E, s);
    // Error of an fp32 score below: expf and the division are within a few
    // units of 2^-24, the softmax's sum of V + 5 roundings adds as many more;
    // one more rounding for the bias.  Twice the bound separates two keys.
    const float eps = (SCORE == QMM_SCORE_SOFTMAX ? 16.f + V : 16.f) * 5.9604645e-8f;
    bool sure = true;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        if (p.bias && e < p.E) s[i] += __ldg(p.bias + e);
        key[i] = e < p.E ? (p.bias ? key_of(s[i]) : key_of(l[i])) : 0u;
    }
    // |s + bias| enters the bound through the rounding of the sum.
    float big = 1.f;
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i < p.E && fabsf(s[i]) < 3e38f) big = fmaxf(big, fabsf(s[i]));
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    }
    const float tol = 2.f * eps * big;
    if (p.n_groups > 1) sure = keep_groups<V, uint32_t, float>(key, s, p, lane, 2.f * tol);
    int mine;
    if (p.bias == nullptr) {
        mine = select_top<V, uint32_t>(key, p.k, p.k, lane, [](int, uint32_t) {});
    } else {
        float last = 0.f;
        mine = select_top<V, uint32_t>(key, p.k, p.k + 1, lane, [&](int j, uint32_t mx) {
            if (mx == 0u) return;  // no candidate left
            const float v = key_value(mx);
            if (j > 0 && last - v <= tol) sure = false;
            last = v;
        });
    }
    if (!sure) mine = route_fp64<T, V, SCORE>(row, p, lane);

    // Weights in fp64, one slot per lane.
    const bool slot = lane < p.k;
    const double NEG = __longlong_as_double(0xfff0000000000000ull);
    const double lj = slot ? (double)Dt<T>::to_f(row[mine]) : NEG;
    double w = 0.0;
    if constexpr (SCORE == QMM_SCORE_SIGMOID) {
        if (slot) w = 1.0 / (1.0 + exp(-lj));
    } else {
        // Relative to the largest chosen logit when renormalised (no score
        // underflows to a zero sum), to the largest of all otherwise.
        double m = lj;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (!p.renormalize) {
            float mf = l[0];
#pragma unroll
            for (int i = 1; i < V; ++i) mf = fmaxf(mf, l[i]);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) mf = fmaxf(mf, __shfl_xor_sync(0xffffffffu, mf, o));
            m = (double)mf;
        }
        if (slot && m != NEG) w = lj == m ? 1.0 : exp(lj - m);
        if (!p.renormalize) {
            double z = 0.0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane + 32 * i < p.E && m != NEG)
                    z += (double)l[i] == m ? 1.0 : (double)expf(l[i] - (float)m);
            z = warp_sum(z);
            w = z > 0.0 ? w / z : 0.0;
        }
    }
    if (p.renormalize) {
        const double sum = warp_sum(w);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (slot) {
        p.indices[t * p.k + lane] = mine;
        p.weights[t * p.k + lane] = nan ? __uint_as_float(0x7fc00000u) : (float)(w * p.scale);
    }
}

template <typename T, int V>
cudaError_t run_route(const RouteArgs &a, cudaStream_t s) {
    RouteParams p{};
    p.logits = a.logits;
    p.bias = a.bias;
    p.indices = a.indices;
    p.weights = a.weights;
    p.T = a.T;
    p.E = a.E;
    p.k = a.top_k;
    p.n_groups = a.n_groups;
    p.topk_groups = a.topk_groups;
    p.group_top = a.group_top;
    p.gsize = a.E / a.n_groups;
    p.renormalize = a.renormalize ? 1 : 0;
    p.scale = a.scale;
    if (p.topk_groups == p.n_groups) p.n_groups = 1;  // every group stays
    const unsigned grid = (unsigned)((a.T + kRouteWarps - 1) / kRouteWarps);
    if (a.score == QMM_SCORE_SIGMOID)
        moe_route_kernel<T, V, QMM_SCORE_SIGMOID><<<grid, 32 * kRouteWarps, 0, s>>>(p);
    else
        moe_route_kernel<T, V, QMM_SCORE_SOFTMAX><<<grid, 32 * kRouteWarps, 0, s>>>(p);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T>
cudaError_t route_size(const RouteArgs &a, cudaStream_t s) {
    const int v = (a.E + 31) / 32;
    if (v <= 1) return run_route<T, 1>(a, s);
    if (v <= 2) return run_route<T, 2>(a, s);
    if (v <= 4) return run_route<T, 4>(a, s);
    if (v <= 8) return run_route<T, 8>(a, s);
    if (v <= 16) return run_route<T, 16>(a, s);
    return run_route<T, 32>(a, s);
}

}  // namespace

cudaError_t launch_moe_route(qmm_dtype dt, const RouteArgs &a, cudaStream_t s) {
    switch (dt) {
    case QMM_F32: return route_size<float>(a, s);
    case QMM_BF16: return route_size<__nv_bfloat16>(a, s);
    default: return route_size<__half>(a, s);
    }
}

}  // namespace qmm
