// Internal declarations of the kernels around the expert products: the router,
// rows in 4 bits, the products of such rows, and the whole layer for a few
// tokens. Not part of the public C ABI (include/moe.h).
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

// MXFP4 rows: 32 consecutive elements share a scale 2^(byte - 127).
struct QuantArgs {
    const void* src;        // quantize: elements; dequantize: values
    bool bf16;              // type of the elements, else fp32
    int64_t blocks;         // of 32 elements, 1 .. kMaxQuantBlocks
    void* values;           // 16 bytes per block
    uint8_t* scales;        // one per block
    void* dst;              // dequantize: elements
};
// Four lanes per block.
constexpr int64_t kMaxQuantBlocks = (int64_t(1) << 30) - 64;
hipError_t launch_quantize_mxfp4(const QuantArgs& a, hipStream_t stream);
hipError_t launch_dequantize_mxfp4(const QuantArgs& a, hipStream_t stream);

// Expert products of 4-bit rows with packed 4-bit weights.
struct ExpertMx4Args {
    bool gated;             // act(g) * u, else the plain product
    const void* rows;       // [max_rows][red / 2]
    const void* row_scales; // [max_rows][red / 32]
    const void* w;          // packed (expert_kernels.h)
    const int32_t* offsets; // [E+1], device
    int32_t E;
    int64_t max_rows;       // 1 .. INT32_MAX
    int32_t red;            // multiple of 32
    int32_t feats;          // features of the output, multiple of 8 (gated: of 16)
    int32_t activation;
    void* out;              // bf16 [max_rows][feats]
    int32_t zero;           // kZeroTail, kZeroHead
};
// Tiles of many rows, or weights streamed for up to 16 rows each; a rule on the
// sizes chooses. The grids are work-items of a launch.
bool expert_mx4_streams(int32_t E, int64_t max_rows, int64_t positions);
// Rows of a tile: 128 from 64 rows per expert on average, unless the tiles
// become too few for the CUs, else 64.
int expert_mx4_tile_rows(bool gated, int32_t E, int64_t max_rows, int32_t feats);
hipError_t launch_expert_mx4(const ExpertMx4Args& a, hipStream_t stream);
int64_t expert_mx4_grid(const ExpertMx4Args& a);
hipError_t launch_expert_mx4_stream(const ExpertMx4Args& a, hipStream_t stream);
int64_t expert_mx4_stream_grid(const ExpertMx4Args& a);

// The whole expert layer for a few tokens.
constexpr int32_t kMaxLayerSlots = 512;
struct LayerArgs {
    const void* x;          // bf16 [T][D]
    const float* scores;    // [T][K]
    const int32_t* ids;     // [T][K]
    int32_t T;              // T K is 1 .. kMaxLayerSlots
    int32_t K;
    int32_t E;
    bool four;              // weights are packed 4-bit, else bf16
    const void* w_gate_up;  // [E][2 F][D]
    const void* w_down;     // [E][D][F]
    int32_t D;              // multiple of 8 (four: of 32)
    int32_t F;              // multiple of 8 (four: of 32)
    int32_t activation;
    void* workspace;        // 4 T K F bytes, F rounded up to 128
    void* y;                // bf16 [T][D]
};
hipError_t launch_few_tokens(const LayerArgs& a, hipStream_t stream);
int64_t few_tokens_grid(const LayerArgs& a);    // work-items of its larger launch

}  // namespace moe
