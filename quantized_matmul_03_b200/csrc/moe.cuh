// moe.cuh -- declarations and device helpers of the mixture-of-experts
// operators: routing (moe_route.cu), the few-row expert products
// (moe_gemv.cu), the grouped tensor-core expert products (moe_tc.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "qmm_internal.cuh"

namespace qmm {

constexpr int kMoeMaxExperts = 1024;  // experts of a router or of a stack
constexpr int kMoeMaxTopK = 32;       // slots per token (one warp lane each)

struct RouteArgs {
    const void *logits;  // [T, E]
    int64_t T;
    int E, top_k;
    const float *bias;  // [E] or null; added to the scores to choose, not to weigh
    int score;          // qmm_score
    int n_groups, topk_groups, group_top;
    bool renormalize;
    double scale;
    int32_t *indices;  // [T, top_k]
    float *weights;    // [T, top_k]
};
cudaError_t launch_moe_route(qmm_dtype dt, const RouteArgs &a, cudaStream_t s);

// One stacked 4-bit weight, [n_experts, rows, cols * 4 / 32] words.
struct ExpertWeight {
    const uint32_t *wq;
    const void *scales, *biases;
};
struct ExpertsArgs {
    const void *x;  // [T, K]
    int64_t T, K;
    const int32_t *indices;  // [T, top_k]
    const float *weights;    // [T, top_k]
    int top_k;
    ExpertWeight gate, up, down;  // [E, I, K], [E, I, K], [E, N, I]
    int64_t n_experts, I, N;
    int group_size, mode, act;
    void *y;  // [T, N]
    void *ws;
};
// Bytes any path of qmm_moe_experts needs for these sizes.
size_t moe_experts_workspace(const ExpertsArgs &a);
// Few rows: two kernels that stream each slot's expert once per slot; more
// tokens than one pass takes go through in blocks.  Supported where a token's
// partial sums of one row fit a CTA's share of shared memory (contractions up to
// 393216 with 32 slots per token).
bool moe_gemv_supported(const ExpertsArgs &a);
size_t moe_gemv_workspace(const ExpertsArgs &a);
cudaError_t launch_moe_gemv(qmm_dtype dt, const ExpertsArgs &a, cudaStream_t s);
// Many rows: sort by expert and two grouped tensor-core products.
bool moe_tc_supported();
size_t moe_tc_workspace(const ExpertsArgs &a);
cudaError_t launch_moe_tc(qmm_dtype dt, const ExpertsArgs &a, cudaStream_t s);

// Gated activation in fp32.
__device__ __forceinline__ float moe_gate(float g, int act) {
    if (act == QMM_ACT_SILU) return g / (1.f + expf(-g));
    // gelu(g) with tanh(z) = 1 - 2 / (1 + e^{2z}): 0.5 g (1 + tanh z) = g (1 - 1 / (1 + e^{2z}))
    const float z = 0.7978845608028654f * (g + 0.044715f * g * g * g);
    return g / (1.f + expf(-2.f * z));
}

// Expert of slot p, or -1 when the slot takes no expert: index -1 leaves the
// slot out, any other index outside [0, E) does too and is reported.
__device__ __forceinline__ int moe_expert(const int32_t *indices, int64_t p, int E, int *err) {
    const int e = indices[p];
    if (e >= 0 && e < E) return e;
    if (e != -1 && err) record_device_error(err, QMM_ERR_INDEX);
    return -1;
}

}  // namespace qmm
