// Host-only stand-ins for the launchers of the router, of 4-bit rows and of the
// layer for a few tokens: each checks that the arguments the host code computed
// are consistent and counts the call; nothing touches the pointers.
#include <cstdio>
#include <cstdlib>

#include "layer_kernels.h"

namespace moe {

int g_route = 0, g_route_grad = 0, g_quant = 0, g_dequant = 0, g_mx4 = 0, g_mx4_stream = 0,
    g_layer = 0;

static void require(bool ok, const char* what) {
    if (!ok) {
        std::fprintf(stderr, "stub: inconsistent launch arguments: %s\n", what);
        std::abort();
    }
}

hipError_t launch_route_topk(const RouteArgs& a, hipStream_t) {
    require(a.T >= 1 && a.K >= 1 && a.E % a.groups == 0 && a.K <= a.E / a.groups * a.kept &&
                a.logits && a.ids && a.scores && (a.sigmoid || !a.bias),
            "route");
    ++g_route;
    return hipSuccess;
}
hipError_t launch_route_topk_grad(const RouteGradArgs& a, hipStream_t) {
    require(a.T >= 1 && a.K >= 1 && a.K <= a.E && a.logits && a.ids && a.grad && a.grad_logits,
            "route gradient");
    ++g_route_grad;
    return hipSuccess;
}
hipError_t launch_quantize_mxfp4(const QuantArgs& a, hipStream_t) {
    require(a.blocks >= 1 && a.blocks <= kMaxQuantBlocks && a.src && a.values && a.scales, "quant");
    ++g_quant;
    return hipSuccess;
}
hipError_t launch_dequantize_mxfp4(const QuantArgs& a, hipStream_t) {
    require(a.blocks >= 1 && a.blocks <= kMaxQuantBlocks && a.dst && a.values && a.scales, "back");
    ++g_dequant;
    return hipSuccess;
}
static void check(const ExpertMx4Args& a) {
    require(a.E >= 1 && a.max_rows >= 1 && a.red % 32 == 0 && a.feats % (a.gated ? 16 : 8) == 0 &&
                a.rows && a.row_scales && a.w && a.offsets && a.out,
            "mx4");
}
hipError_t launch_expert_mx4(const ExpertMx4Args& a, hipStream_t) {
    check(a);
    ++g_mx4;
    return hipSuccess;
}
hipError_t launch_expert_mx4_stream(const ExpertMx4Args& a, hipStream_t) {
    check(a);
    ++g_mx4_stream;
    return hipSuccess;
}
int64_t expert_mx4_grid(const ExpertMx4Args& a) { return a.max_rows + a.feats; }
int64_t expert_mx4_stream_grid(const ExpertMx4Args& a) { return a.max_rows + a.feats; }
hipError_t launch_few_tokens(const LayerArgs& a, hipStream_t) {
    require(a.T >= 1 && a.K >= 1 && a.T * a.K <= kMaxLayerSlots && a.D % (a.four ? 32 : 8) == 0 &&
                a.F % (a.four ? 32 : 8) == 0 && a.workspace && a.y,
            "layer");
    ++g_layer;
    return hipSuccess;
}
int64_t few_tokens_grid(const LayerArgs& a) { return int64_t(a.T) * a.F; }

}  // namespace moe
