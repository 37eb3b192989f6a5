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

static_assert(MOE_MAX_LAYER_SLOTS == moe::kMaxLayerSlots &&
                  MOE_MAX_ROUTE_GROUPS == moe::kMaxRouteGroups,
              "the kernels' limits");

namespace {

using moe::activation_ok;
using moe::apart;
using moe::experts_ok;
using moe::Input;
using moe::kZeroFlags;
using moe::misaligned;
using moe::offsets_of;
using moe::status_of;
using moe::weights_of;
using moe::width_ok;
using moe::zero_of;

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

int run_quant(bool back, const void* from, int32_t dtype, int64_t rows, int32_t width, void* values,
              void* scales, void* to, void* stream) {
    if ((dtype != MOE_F32 && dtype != MOE_BF16) || rows < 0 || width < 32 ||
        width > MOE_MAX_GEMM_WIDTH || width % 32 != 0 ||
        rows > moe::kMaxQuantBlocks / (width / 32))
        return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    const void* elements = back ? to : from;
    if (!elements || !values || !scales || misaligned(elements, 16) || misaligned(values, 16))
        return MOE_ERR_INVALID_ARG;
    const int64_t blocks = rows * (width / 32);
    const Input x = {elements, blocks * 32 * (dtype == MOE_F32 ? 4 : 2)};
    const Input v = {values, blocks * 16}, s = {scales, blocks};
    if (back ? !apart(to, x.bytes, {v, s}) : !apart(values, v.bytes, {x, s}) ||
                                                 !apart(scales, s.bytes, {x}))
        return MOE_ERR_INVALID_ARG;
    moe::QuantArgs a;
    a.src = from;
    a.bf16 = dtype == MOE_BF16;
    a.blocks = blocks;
    a.values = values;
    a.scales = static_cast<uint8_t*>(scales);
    a.dst = to;
    return status_of(back ? moe::launch_dequantize_mxfp4(a, static_cast<hipStream_t>(stream))
                          : moe::launch_quantize_mxfp4(a, static_cast<hipStream_t>(stream)));
}

int run_mx4(bool gated, const void* values, const void* row_scales, const void* packed,
            const int32_t* offsets, int32_t E, int64_t max_rows, int32_t red, int32_t feats,
            int32_t activation, void* out, int32_t flags, void* stream) {
    const int64_t packed_bytes = moe_mxfp4_weights_bytes(E, gated ? 2 * feats : feats, red);
    if (packed_bytes < 0 || max_rows < 0 || max_rows > INT32_MAX || (flags & ~kZeroFlags))
        return MOE_ERR_INVALID_ARG;
    if (max_rows == 0) return MOE_OK;
    if (!values || !row_scales || !packed || !offsets || !out || misaligned(values, 16) ||
        misaligned(packed, 16) || misaligned(offsets, 4) || misaligned(out, 16) ||
        !apart(out, max_rows * feats * 2,
               {{values, max_rows * (red / 2)}, {row_scales, max_rows * (red / 32)},
                {packed, packed_bytes}, offsets_of(offsets, E)}))
        return MOE_ERR_INVALID_ARG;
    moe::ExpertMx4Args a;
    a.gated = gated;
    a.rows = values;
    a.row_scales = row_scales;
    a.w = packed;
    a.offsets = offsets;
    a.E = E;
    a.max_rows = max_rows;
    a.red = red;
    a.feats = feats;
    a.activation = activation;
    a.out = out;
    a.zero = zero_of(flags);
    if (moe::expert_mx4_streams(E, max_rows, gated ? int64_t(2) * feats : feats)) {
        if (moe::expert_mx4_stream_grid(a) > moe::kMaxGrid) return MOE_ERR_INVALID_ARG;
        return status_of(moe::launch_expert_mx4_stream(a, static_cast<hipStream_t>(stream)));
    }
    if (moe::expert_mx4_grid(a) > moe::kMaxGrid) return MOE_ERR_INVALID_ARG;
    return status_of(moe::launch_expert_mx4(a, static_cast<hipStream_t>(stream)));
}

}  // namespace

namespace moe {

// Where the form that streams the weights (16-row tiles, the sum split over a
// workgroup's wavefronts) is the faster one. Measured on MI355X with other weights
// in every call, streamed against tiled:
//   - up to 8 rows per expert: 64 experts of 7168 -> 2 x 2048 145 and 171 us at 8
//     rows each, 230 and 173 at 16; 256 of 2048 -> 7168 315 and 346, 465 and 360.
//   - while its workgroups are few (the tiled form then leaves CUs idle): one expert
//     of 4096 -> 2 x 2048 18.5 and 21.9 us at 256 rows (1024 workgroups), 31.3 and
//     22.1 at 512 (2048); one of 2048 -> 7168 12.4 and 13.5 at 128 (896), 20.1 and
//     14.0 at 256 (1792); 24 of 1984 -> 1000 12.5 and 14.4 at 768 (768), 19.7 and
//     15.6 at 1536 (1536).
bool expert_mx4_streams(int32_t E, int64_t max_rows, int64_t positions) {
    if (max_rows <= int64_t(8) * E) return true;
    const int64_t experts = max_rows < E ? max_rows : E;
    const int64_t tiles = (max_rows + 15) / 16;
    return (positions + 63) / 64 * (tiles > experts ? tiles : experts) <= 1024;
}

}  // namespace moe

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

int moe_quantize_mxfp4(const void* d_x, int32_t dtype, int64_t rows, int32_t width, void* d_values,
                       void* d_scales, void* stream) {
    return run_quant(false, d_x, dtype, rows, width, d_values, d_scales, nullptr, stream);
}

int moe_dequantize_mxfp4(const void* d_values, const void* d_scales, int32_t dtype, int64_t rows,
                         int32_t width, void* d_x, void* stream) {
    return run_quant(true, nullptr, dtype, rows, width, const_cast<void*>(d_values),
                     const_cast<void*>(d_scales), d_x, stream);
}

int moe_grouped_gemm_mxfp4_rows(const void* d_values, const void* d_scales, const void* d_packed,
                                const int32_t* d_offsets, int32_t num_experts, int64_t max_rows,
                                int32_t k_in, int32_t n_out, void* d_out, int32_t flags,
                                void* stream) {
    return run_mx4(false, d_values, d_scales, d_packed, d_offsets, num_experts, max_rows, k_in,
                   n_out, MOE_ACT_SILU, d_out, flags, stream);
}

int moe_gated_grouped_gemm_mxfp4_rows(const void* d_values, const void* d_scales,
                                      const void* d_packed, const int32_t* d_offsets,
                                      int32_t num_experts, int64_t max_rows, int32_t k_in,
                                      int32_t n_hidden, int32_t activation, void* d_h,
                                      int32_t flags, void* stream) {
    if (!width_ok(n_hidden, 16) || n_hidden > MOE_MAX_GEMM_WIDTH / 2 || !activation_ok(activation))
        return MOE_ERR_INVALID_ARG;
    return run_mx4(true, d_values, d_scales, d_packed, d_offsets, num_experts, max_rows, k_in,
                   n_hidden, activation, d_h, flags, stream);
}

int64_t moe_few_tokens_workspace_bytes(int32_t T, int32_t K, int32_t n_hidden) {
    if (T < 0 || K < 1 || K > MOE_MAX_TOPK || T > MOE_MAX_LAYER_SLOTS / K || !width_ok(n_hidden, 8) ||
        n_hidden > MOE_MAX_GEMM_WIDTH / 2)
        return -1;
    return int64_t(T) * K * ((n_hidden + 127) / 128 * 128) * 4;
}

int moe_few_tokens_layer(const void* d_x, const float* d_topk_scores, const int32_t* d_topk_ids,
                         int32_t T, int32_t K, const void* d_w_gate_up, const void* d_w_down,
                         int32_t weight_layout, int32_t num_experts, int32_t hidden,
                         int32_t n_hidden, int32_t activation, void* d_workspace,
                         int64_t workspace_bytes, void* d_y, void* stream) {
    const bool four = weight_layout == MOE_WEIGHTS_MXFP4;
    const int64_t need = moe_few_tokens_workspace_bytes(T, K, n_hidden);
    if (need < 0 || (!four && weight_layout != MOE_WEIGHTS_ROW_MAJOR) || !experts_ok(num_experts) ||
        !width_ok(hidden, four ? 32 : 8) || !width_ok(n_hidden, four ? 32 : 8) ||
        !activation_ok(activation))
        return MOE_ERR_INVALID_ARG;
    Input w1 = weights_of(d_w_gate_up, num_experts, int64_t(2) * n_hidden, hidden);
    Input w2 = weights_of(d_w_down, num_experts, hidden, n_hidden);
    if (four) {
        w1.bytes = moe_mxfp4_weights_bytes(num_experts, 2 * n_hidden, hidden);
        w2.bytes = moe_mxfp4_weights_bytes(num_experts, hidden, n_hidden);
        if (w1.bytes < 0 || w2.bytes < 0) return MOE_ERR_INVALID_ARG;
    }
    if (T == 0) return MOE_OK;
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
    if (!d_x || !d_topk_scores || !d_topk_ids || !d_w_gate_up || !d_w_down || !d_workspace ||
        !d_y || misaligned(d_x, 16) || misaligned(d_topk_scores, 4) || misaligned(d_topk_ids, 4) ||
        misaligned(d_w_gate_up, 16) || misaligned(d_w_down, 16) || misaligned(d_workspace, 16) ||
        misaligned(d_y, 16))
        return MOE_ERR_INVALID_ARG;
    const Input x = {d_x, int64_t(T) * hidden * 2};
    const Input s = {d_topk_scores, int64_t(T) * K * 4}, ids = {d_topk_ids, int64_t(T) * K * 4};
    if (!apart(d_workspace, need, {x, s, ids, w1, w2}) ||
        !apart(d_y, x.bytes, {x, s, ids, w1, w2, {d_workspace, need}}))
        return MOE_ERR_INVALID_ARG;
    moe::LayerArgs a;
    a.x = d_x;
    a.scores = d_topk_scores;
    a.ids = d_topk_ids;
    a.T = T;
    a.K = K;
    a.E = num_experts;
    a.four = four;
    a.w_gate_up = d_w_gate_up;
    a.w_down = d_w_down;
    a.D = hidden;
    a.F = n_hidden;
    a.activation = activation;
    a.workspace = d_workspace;
    a.y = d_y;
    if (moe::few_tokens_grid(a) > moe::kMaxGrid) return MOE_ERR_INVALID_ARG;
    return status_of(moe::launch_few_tokens(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
