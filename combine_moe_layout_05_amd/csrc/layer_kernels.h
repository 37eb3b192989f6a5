// Internal declarations of the kernels around the expert products: the router.
// Not part of the public C ABI (include/moe.h).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace moe {

constexpr int32_t kMaxRouteGroups = 64;      // one lane each

struct RouteArgs {
    const void* logits;     // [T][E] fp32 or bf16
    bool bf16;
    const float* bias;      // [E] or null (sigmoid only)
    int32_t T;              // >= 1
    int32_t E;              // 1 .. 1024
    int32_t K;              // 1 .. min(16, E)
    bool sigmoid;
    bool renormalize;
    float scale;
    int32_t groups;         // divides E, 1 .. kMaxRouteGroups
    int32_t kept;           // 1 .. groups
    int32_t* ids;           // [T][K]
    float* scores;          // [T][K]
};
hipError_t launch_route_topk(const RouteArgs& a, hipStream_t stream);

struct RouteGradArgs {
    const void* logits;     // as above
    bool bf16;
    const int32_t* ids;     // [T][K]
    const float* grad;      // [T][K], of the scores
    int32_t T;
    int32_t E;
    int32_t K;
    bool sigmoid;
    bool renormalize;
    float scale;
    void* grad_logits;      // [T][E], the logits' type
};
hipError_t launch_route_topk_grad(const RouteGradArgs& a, hipStream_t stream);

}  // namespace moe
