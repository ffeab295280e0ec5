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
// One warp per token, lane l holding V neighbouring experts (V = 1, 2, 4 .. 32).
// The top_k-th largest of the 32 lanes' maxima bounds the top_k-th largest key
// from below; the few keys that reach it (about top_k + 2) are packed into
// shared memory and each finds its rank by counting the better ones.  (A
// maximum, an index and a search of the owner's keys per chosen expert, the
// form kept for tokens with more than 32 keys at the bound, took 47 us for
// 16384 tokens of 256 experts where this takes 36 us.)  Groups that are a
// power-of-two number of lanes wide find their two best by exchanges within
// those lanes, all groups at once; other groups one after the other.  A warp
// of a long batch takes several tokens and computes their weights together, a
// slot per lane.  The kernel reads the logits once and writes 8 bytes per slot;
// small batches are bound by the launch, long ones by instruction issue.
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

constexpr int kRouteWarps = 8;  // tokens per CTA

struct RouteParams {
    const void *logits;
    const float *bias;
    int32_t *indices;
    float *weights;
    int64_t T;
    int E, k, n_groups, topk_groups, group_top, gsize;
    int group_lanes;  // lanes of a group when that is a power of two, else 0
    int vec;          // logits rows in whole aligned 16-byte units
    int kp_log;       // slots of a token padded to 2^kp_log lanes
    int tokens;       // tokens of a warp (at most 32 >> kp_log)
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

// The k best of key[V] (lane l: experts V l + i); lane j returns the j-th
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
        const uint32_t at = __reduce_min_sync(0xffffffffu, best == mx ? (uint32_t)(lane * V + bi) : 0xffffffffu);
        if (j < k && lane == j) mine = (int)at;
        check(j, mx);
        if (at / V == (uint32_t)lane) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == bi) key[i] = 0;
            rescan();
        }
    }
    return mine;
}

// The lane's V logits of a row, -inf past the last expert.
template <typename T, int V>
__device__ __forceinline__ void load_logits(const T *row, int E, bool vec, int lane, float (&l)[V]) {
    constexpr int U = 16 / (int)sizeof(T);  // logits of 16 bytes
    if constexpr (V >= U) {
        if (vec) {
#pragma unroll
            for (int c = 0; c < V / U; ++c) {
                const bool in = lane * V + c * U < E;  // E is a multiple of U here
                const uint4 r = in ? *reinterpret_cast<const uint4 *>(row + lane * V + c * U) : make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                for (int i = 0; i < U; ++i)
                    l[c * U + i] = in ? Dt<T>::to_f(reinterpret_cast<const T *>(w)[i]) : __uint_as_float(0xff800000u);
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        l[i] = e < E ? Dt<T>::to_f(row[e]) : __uint_as_float(0xff800000u);
    }
}

template <int V, typename F, int SCORE>
__device__ __forceinline__ void scores_of(const float (&l)[V], int lane, int E, F (&s)[V]) {
    if constexpr (SCORE == QMM_SCORE_SIGMOID) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (std::is_same<F, double>::value) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
            else s[i] = __fdividef(1.f, 1.f + __expf(-l[i]));
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
            // whose logits are all -inf has no terms.  A NaN logit has a NaN
            // score and is left out of the sum, as out of the maximum, so that
            // the others keep their order.
            if (m == __uint_as_float(0xff800000u)) s[i] = l[i] == l[i] ? F(0) : F(l[i]);
            else if (l[i] == m) s[i] = 1;
            else if constexpr (std::is_same<F, double>::value) s[i] = exp((double)l[i] - (double)m);
            else s[i] = __expf(l[i] - m);
            if (lane * V + i < E && s[i] == s[i]) z += s[i];
        }
        z = warp_sum(z);
        const F inv = z > 0 ? F(1) / z : F(0);
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = std::is_same<F, double>::value && z > 0 ? s[i] / z : s[i] * inv;
    }
}

// Candidates of the best groups: clears the keys of every other group.  sel:
// the values groups are scored by.  Returns false if the last group kept and
// the best one left out lie within tol of each other.
template <int V, typename Key, typename F>
__device__ __forceinline__ bool keep_groups(Key (&key)[V], const F (&sel)[V], const RouteParams &p, int lane,
                                            F tol) {
    const int G = p.n_groups;
    if (p.group_lanes > 0) {
        // Every lane's experts belong to one group: its two best, then the
        // group's by exchanges over its lanes (a total order on (key, index) is
        // not needed: equal keys have equal values).
        Key b1 = 0, b2 = 0;
        F v1 = 0, v2 = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Key q = lane * V + i < p.E ? key_of(sel[i]) : Key(0);
            if (q > b1) {
                b2 = b1; v2 = v1;
                b1 = q; v1 = sel[i];
            } else if (q > b2) {
                b2 = q; v2 = sel[i];
            }
        }
        for (int o = 1; o < p.group_lanes; o <<= 1) {
            const Key c1 = __shfl_xor_sync(0xffffffffu, b1, o), c2 = __shfl_xor_sync(0xffffffffu, b2, o);
            const F w1 = __shfl_xor_sync(0xffffffffu, v1, o), w2 = __shfl_xor_sync(0xffffffffu, v2, o);
            if (c1 > b1) {
                const bool mid = b1 > c2;
                b2 = mid ? b1 : c2; v2 = mid ? v1 : w2;
                b1 = c1; v1 = w1;
            } else if (c1 > b2) {
                b2 = c1; v2 = w1;
            }
        }
        const F score = p.group_top == 2 && p.gsize > 1 ? v1 + v2 : v1;
        const int g = lane / p.group_lanes;
        const Key mine = g < G ? key_of(score) : Key(0);
        int rank = 0;
        for (int o = 0; o < G; ++o) {
            const Key c = __shfl_sync(0xffffffffu, mine, o * p.group_lanes);
            rank += (c > mine || (c == mine && o < g)) ? 1 : 0;
        }
        const bool live = rank < p.topk_groups;
        // The scores of the last group kept and the best one left out.
        const unsigned lk = __ballot_sync(0xffffffffu, g < G && rank == p.topk_groups - 1);
        const unsigned lo = __ballot_sync(0xffffffffu, g < G && rank == p.topk_groups);
        const F last = __shfl_sync(0xffffffffu, score, lk ? __ffs(lk) - 1 : 0);
        const F next = __shfl_sync(0xffffffffu, score, lo ? __ffs(lo) - 1 : 0);
        if (!live) {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = 0;
        }
        return !(lo && last - next <= tol);
    }
    Key mine = 0;  // lane g: group g's score as a key
    F mine_v = 0;
    for (int g = 0; g < G; ++g) {
        Key b1 = 0, b2 = 0;
        F v1 = 0, v2 = 0;
        bool h2 = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
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
        const int e = lane * V + i;
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
        const int e = lane * V + i;
        l[i] = e < p.E ? Dt<T>::to_f(row[e]) : __uint_as_float(0xff800000u);
    }
    scores_of<V, double, SCORE>(l, lane, p.E, s);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        if (p.bias && e < p.E) s[i] += (double)__ldg(p.bias + e);
        key[i] = e < p.E ? (p.bias ? key_of(s[i]) : key_of((double)l[i])) : 0ull;
    }
    if (p.n_groups > 1) keep_groups<V, uint64_t, double>(key, s, p, lane, -1.0);
    return select_top<V, uint64_t>(key, p.k, p.k, lane, [](int, uint64_t) {});
}

// Shared memory of one warp.
struct WarpBox {
    uint2 cand[32];     // keys at the bound and their experts
    uint32_t order[34]; // the best keys in order
    int32_t chosen[32]; // experts of the warp's slots
};

// The k best of key[V] into out[0..k); false if the fp32 order of two
// neighbours (the first left out included, when `check`) is in doubt.
template <int V>
__device__ __forceinline__ bool select_ranked(uint32_t (&key)[V], int k, bool check, float tol, int lane,
                                              WarpBox &box, int32_t *out) {
    uint32_t top = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = max(top, key[i]);
    const int want = check ? k + 1 : k;
    uint32_t bound = 0, m = top;
    for (int j = 0; j < want; ++j) {
        bound = __reduce_max_sync(0xffffffffu, m);
        if (m == bound) m = 0;  // (equal maxima leave together: the bound only gets lower)
    }
    bound = max(bound, 1u);
    int n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const bool in = key[i] >= bound;
        const unsigned who = __ballot_sync(0xffffffffu, in);
        const int at = n + __popc(who & ((1u << lane) - 1u));
        if (in && at < 32) box.cand[at] = make_uint2(key[i], (uint32_t)(lane * V + i));
        n += __popc(who);
    }
    __syncwarp();
    if (n > 32 || want > 32) {
        float last = 0.f;
        bool sure = true;
        const int mine = select_top<V, uint32_t>(key, k, want, lane, [&](int j, uint32_t mx) {
            if (!check || mx == 0u) return;  // (0: no candidate left)
            const float v = key_value(mx);
            if (j > 0 && last - v <= tol) sure = false;
            last = v;
        });
        if (lane < k) out[lane] = mine;
        __syncwarp();
        return sure;
    }
    const uint2 c = lane < n ? box.cand[lane] : make_uint2(0u, 0u);
    int rank = 0;
    for (int j = 0; j < n; ++j) {
        const uint2 o = box.cand[j];
        rank += (o.x > c.x || (o.x == c.x && o.y < c.y)) ? 1 : 0;
    }
    if (lane < n && rank < want) {
        box.order[rank] = c.x;
        if (rank < k) out[rank] = (int32_t)c.y;
    }
    __syncwarp();
    bool doubt = false;
    if (check && lane + 1 < min(n, want)) doubt = key_value(box.order[lane]) - key_value(box.order[lane + 1]) <= tol;
    return !__any_sync(0xffffffffu, doubt);
}

template <typename T, int V, int SCORE>
__global__ void __launch_bounds__(32 * kRouteWarps, V <= 8 ? 4 : 2) moe_route_kernel(const RouteParams p) {
    __shared__ WarpBox boxes[kRouteWarps];
    const int lane = threadIdx.x & 31;
    WarpBox &box = boxes[threadIdx.x >> 5];
    const int64_t t0 = ((int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5)) * p.tokens;
    if (t0 >= p.T) return;
    const int count = (int)min((int64_t)p.tokens, p.T - t0);
    const T *rows = static_cast<const T *>(p.logits) + t0 * p.E;
    const int kp = 1 << p.kp_log, q = lane >> p.kp_log, j = lane & (kp - 1);  // this lane's token and slot
    const double NEG = __longlong_as_double(0xfff0000000000000ull);
    bool my_nan = false;
    double my_max = NEG, my_z = 0.0;

    for (int i0 = 0; i0 < count; ++i0) {
        const T *row = rows + (int64_t)i0 * p.E;
        float l[V];
        bool nan = false;
        load_logits<T, V>(row, p.E, p.vec != 0, lane, l);
#pragma unroll
        for (int i = 0; i < V; ++i) nan = nan || l[i] != l[i];
        nan = __any_sync(0xffffffffu, nan);

        uint32_t key[V];
        float s[V];
        if (p.bias != nullptr || p.n_groups > 1) scores_of<V, float, SCORE>(l, lane, p.E, s);
        // Error of an fp32 score: __expf is within 2 + 1.2 |x| units of 2^-23 of
        // its value, which times the score (sigmoid: times s (1 - s) |x| < 0.23)
        // stays below 8 units of 2^-24; the softmax's divisor adds the mean of
        // the same over its terms (|x| below ln E on average) and V + 5
        // roundings; the division two; one more rounding for the bias.  Twice
        // the bound separates two keys.
        constexpr float eps = (SCORE == QMM_SCORE_SOFTMAX ? 40.f + V : 16.f) * 5.9604645e-8f;
        bool sure = true;
        float big = 1.f;  // |s + bias| enters the bound through the rounding of the sum
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
            if (p.bias && e < p.E) {
                s[i] += __ldg(p.bias + e);
                if (fabsf(s[i]) < 3e38f) big = fmaxf(big, fabsf(s[i]));
            }
            key[i] = e < p.E ? (p.bias ? key_of(s[i]) : key_of(l[i])) : 0u;
        }
        if (p.bias) big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));  // (positive)
        const float tol = 2.f * eps * big;
        if (p.n_groups > 1) sure = keep_groups<V, uint32_t, float>(key, s, p, lane, 2.f * tol);
        int32_t *out = box.chosen + i0 * kp;
        if (!select_ranked<V>(key, p.k, p.bias != nullptr, tol, lane, box, out)) sure = false;
        if (!sure) {
            const int mine = route_fp64<T, V, SCORE>(row, p, lane);
            __syncwarp();
            if (lane < p.k) out[lane] = mine;
        }
        if (q == i0) my_nan = nan;
        if (SCORE == QMM_SCORE_SOFTMAX && !p.renormalize) {
            // The largest logit and the sum over all experts relative to it: terms
            // and a lane's V additions in fp32, at most V + 8 units of 2^-24 off
            // (expf 2, its argument ln E in the mean), the 32 lanes in fp64.
            float m = l[0];
#pragma unroll
            for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            float z = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane * V + i < p.E && m != __uint_as_float(0xff800000u)) z += l[i] == m ? 1.f : expf(l[i] - m);
            const double zd = warp_sum((double)z);
            if (q == i0) {
                my_max = (double)m;
                my_z = zd;
            }
        }
        __syncwarp();
    }

    // Weights of all of the warp's slots at once, in fp64.
    const bool slot = q < count && j < p.k;
    const int e = slot ? box.chosen[lane] : 0;
    const double lj = slot ? (double)Dt<T>::to_f(rows[(int64_t)q * p.E + e]) : NEG;
    double w = 0.0;
    if constexpr (SCORE == QMM_SCORE_SIGMOID) {
        if (slot) {
            const double x = exp(-fabs(lj));
            w = (lj >= 0.0 ? 1.0 : x) / (1.0 + x);
            if (lj != lj) w = lj;
        }
    } else {
        // Relative to the largest chosen logit when renormalised (no score
        // underflows to a zero sum), to the largest of all otherwise.
        double m = my_max;
        if (p.renormalize) {
            m = lj;
            for (int o = kp >> 1; o >= 1; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
        }
        if (slot && m != NEG) w = lj == m ? 1.0 : exp(lj - m);
        if (!p.renormalize) w = my_z > 0.0 ? w / my_z : 0.0;
    }
    if (p.renormalize) {
        double sum = w;
        for (int o = kp >> 1; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (slot) {
        const int64_t at = (t0 + q) * p.k + j;
        p.indices[at] = e;
        p.weights[at] = my_nan ? __uint_as_float(0x7fc00000u) : (float)(w * p.scale);
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
    const int gl = p.gsize % V == 0 ? p.gsize / V : 0;
    p.group_lanes = (gl & (gl - 1)) == 0 ? gl : 0;
    p.vec = (a.E * sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0;
    p.renormalize = a.renormalize ? 1 : 0;
    p.scale = a.scale;
    if (p.topk_groups == p.n_groups) p.n_groups = 1;  // every group stays
    while ((1 << p.kp_log) < p.k) ++p.kp_log;
    // Several tokens per warp once there are enough for every SM to stay full
    // (32 warps each).
    p.tokens = 32 >> p.kp_log;
    while (p.tokens > 1 && a.T < (int64_t)num_sms() * 32 * p.tokens) p.tokens >>= 1;
    const int64_t per = (int64_t)kRouteWarps * p.tokens;
    const unsigned grid = (unsigned)((a.T + per - 1) / per);
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
