// C ABI entry points of what lies around the expert products (include/moe.h):
// host argument checks and the choice of kernel. No entry point touches the
// device before every check has passed.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "api_checks.h"
#include "layer_kernels.h"
#include "moe.h"

namespace {

using moe::apart;
using moe::experts_ok;
using moe::Input;
using moe::misaligned;
using moe::status_of;

bool route_ok(int32_t dtype, int32_t T, int32_t E, int32_t K, int32_t score, int32_t flags,
              float scale) {
    // A wavefront per token.
    return (dtype == MOE_F32 || dtype == MOE_BF16) && T >= 0 && int64_t(T) * 64 <= moe::kMaxGrid &&
           experts_ok(E) && K >= 1 && K <= MOE_MAX_TOPK && K <= E &&
           (score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID) &&
           !(flags & ~MOE_ROUTE_RENORMALIZE) && std::isfinite(scale);
}

Input logits_of(const void* p, int32_t dtype, int64_t T, int64_t E) {
    return {p, T * E * (dtype == MOE_F32 ? 4 : 2)};
}

}  // namespace

extern "C" {

int moe_route_topk(const void* d_logits, int32_t dtype, const float* d_bias, int32_t T, int32_t E,
                   int32_t K, int32_t score, int32_t flags, float scale, int32_t num_groups,
                   int32_t topk_groups, int32_t* d_ids, float* d_scores, void* stream) {
    if (!route_ok(dtype, T, E, K, score, flags, scale) || num_groups < 1 ||
        num_groups > moe::kMaxRouteGroups || E % num_groups != 0 || topk_groups < 1 ||
        topk_groups > num_groups || K > E / num_groups * topk_groups ||
        (d_bias && score != MOE_SCORE_SIGMOID))
        return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!d_logits || !d_ids || !d_scores || misaligned(d_logits, dtype == MOE_F32 ? 4 : 2) ||
        misaligned(d_bias, 4) || misaligned(d_ids, 4) || misaligned(d_scores, 4))
        return MOE_ERR_INVALID_ARG;
    const Input logits = logits_of(d_logits, dtype, T, E);
    const Input bias = {d_bias, d_bias ? int64_t(E) * 4 : 0};
    const int64_t out = int64_t(T) * K * 4;
    if (!apart(d_ids, out, {logits, bias}) || !apart(d_scores, out, {logits, bias, {d_ids, out}}))
        return MOE_ERR_INVALID_ARG;
    moe::RouteArgs a;
    a.logits = d_logits;
    a.bf16 = dtype == MOE_BF16;
    a.bias = d_bias;
    a.T = T;
    a.E = E;
    a.K = K;
    a.sigmoid = score == MOE_SCORE_SIGMOID;
    a.renormalize = (flags & MOE_ROUTE_RENORMALIZE) != 0;
    a.scale = scale;
    a.groups = num_groups;
    a.kept = topk_groups;
    a.ids = d_ids;
    a.scores = d_scores;
    return status_of(moe::launch_route_topk(a, static_cast<hipStream_t>(stream)));
}

int moe_route_topk_backward(const void* d_logits, int32_t dtype, const int32_t* d_ids,
                            const float* d_grad_scores, int32_t T, int32_t E, int32_t K,
                            int32_t score, int32_t flags, float scale, void* d_grad_logits,
                            void* stream) {
    if (!route_ok(dtype, T, E, K, score, flags, scale)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    const uintptr_t align = dtype == MOE_F32 ? 4 : 2;
    if (!d_logits || !d_ids || !d_grad_scores || !d_grad_logits || misaligned(d_logits, align) ||
        misaligned(d_grad_logits, align) || misaligned(d_ids, 4) || misaligned(d_grad_scores, 4))
        return MOE_ERR_INVALID_ARG;
    const Input logits = logits_of(d_logits, dtype, T, E);
    const int64_t slots = int64_t(T) * K * 4;
    if (!apart(d_grad_logits, logits.bytes, {logits, {d_ids, slots}, {d_grad_scores, slots}}))
        return MOE_ERR_INVALID_ARG;
    moe::RouteGradArgs a;
    a.logits = d_logits;
    a.bf16 = dtype == MOE_BF16;
    a.ids = d_ids;
    a.grad = d_grad_scores;
    a.T = T;
    a.E = E;
    a.K = K;
    a.sigmoid = score == MOE_SCORE_SIGMOID;
    a.renormalize = (flags & MOE_ROUTE_RENORMALIZE) != 0;
    a.scale = scale;
    a.grad_logits = d_grad_logits;
    return status_of(moe::launch_route_topk_grad(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
