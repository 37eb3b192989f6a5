// Internal declarations of the expert feed-forward kernels: the gated block's
// products, their backward, and the products with 4-bit weights. Not part of
// the public C ABI (include/moe.h).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace moe {

// What an expert product writes.
//   kPlain       out[r][n] = sum over k of rows[r][k] * w[e][n][k]
//   kGated       the weight holds 2F rows, gate then up: out[r][f] =
//                act(g) * u, optionally pre[r] = [g | u]
//   kInputGrad   out[r][k] = sum over n of rows[r][n] * w[e][n][k]
//   kGatedGrad   the same sum as dh, then out[r] = [dh*u*act'(g) | dh*act(g)]
//                from pre[r] = [g | u]
enum class ExpertOp { kPlain, kGated, kInputGrad, kGatedGrad };

// Tiles or steps of `size` rows that `rows` (0 .. INT32_MAX) rows take. The sum
// is formed in 32 unsigned bits, which it stays within.
__host__ __device__ constexpr int32_t expert_row_parts(int32_t rows, uint32_t size) {
    return static_cast<int32_t>((static_cast<uint32_t>(rows) + size - 1) / size);
}

// Rows a product sets to +0.0 beside the ones it computes.
constexpr int32_t kZeroTail = 1;        // from offsets[E] on
constexpr int32_t kZeroHead = 2;        // before offsets[0]

struct ExpertGemmArgs {
    ExpertOp op;
    const void* rows;       // bf16 [max_rows][red]
    const void* w;          // bf16 [E][n][k] as the operation reads it
    const int32_t* offsets; // [E+1], device
    int32_t E;
    int64_t max_rows;       // 1 .. INT32_MAX
    int32_t red;            // length of the sums, multiple of 8
    int32_t feats;          // features of the output (F for kGated), multiple of 8
    int32_t activation;     // moe_activation
    void* out;              // bf16 [max_rows][feats], kGatedGrad: [max_rows][2 feats]
    float* pre;             // [max_rows][2 feats] or null
    int32_t zero;           // kZeroTail, kZeroHead: rows outside the segments that get +0.0
};
// Whether it runs in the small tiles, by a rule on the sizes.
bool expert_small_tile(ExpertOp op, int32_t E, int64_t max_rows, int32_t feats);
hipError_t launch_expert_gemm(const ExpertGemmArgs& a, hipStream_t stream);
// Work-items such a launch takes (workgroups times their threads); at most
// kMaxGrid of them fit a launch.
constexpr int64_t kMaxGrid = UINT32_MAX;
int64_t expert_gemm_grid(const ExpertGemmArgs& a);

struct ExpertWgradArgs {
    const void* dy;         // bf16 [max_rows][N]
    const void* x;          // bf16 [max_rows][K]
    const int32_t* offsets; // [E+1], device
    int32_t E;
    int64_t max_rows;       // 0 .. INT32_MAX
    int32_t N;              // multiple of 8
    int32_t K;              // multiple of 8
    bool f32;               // element type of dw: fp32, else bf16
    bool accumulate;        // add to what dw holds
    void* dw;               // [E][N][K]
};
hipError_t launch_expert_wgrad(const ExpertWgradArgs& a, hipStream_t stream);
int64_t expert_wgrad_grid(const ExpertWgradArgs& a);

// Packed 4-bit weights: for 16-feature block b and 128-k step t one KiB, lane
// l's 16 bytes being feature 16b + l % 16, dword s (0..3) the 8 values of k =
// 128t + 32s + 8 (l / 16) .. + 8 (the A fragment of the matrix-core product
// over the 32 k of scale group s). After all values, for each (b, t) the 16
// features' scales of the step's 4 groups, a dword each. Features past N and
// k past K hold zeros with scale 1.
constexpr int32_t kMxfp4Step = 128;
inline int64_t mxfp4_tiles(int32_t E, int32_t N, int32_t K) {
    return int64_t(E) * ((int64_t(N) + 15) / 16) * ((int64_t(K) + kMxfp4Step - 1) / kMxfp4Step);
}
inline int64_t mxfp4_bytes(int32_t E, int32_t N, int32_t K) { return mxfp4_tiles(E, N, K) * 1088; }
struct PackMxfp4Args {
    const void* blocks;     // uint8 [E][N][K/2]
    const void* scales;     // uint8 [E][N][K/32]
    int32_t E;
    int32_t N;
    int32_t K;              // multiple of 32
    void* dst;              // mxfp4_bytes(E, N, K)
};
// Work-items of the packing launch: one per feature of a block and step.
inline int64_t mxfp4_pack_grid(int32_t E, int32_t N, int32_t K) {
    return (mxfp4_tiles(E, N, K) * 16 + 255) / 256 * 256;
}
hipError_t launch_pack_mxfp4(const PackMxfp4Args& a, hipStream_t stream);

// Products for few rows per expert: the weights are streamed once from HBM
// straight into fragment registers, the sum split over a workgroup's
// wavefronts.
struct ExpertStreamArgs {
    bool mxfp4;             // w is packed 4-bit, else bf16 [E][n][red]
    bool gated;             // act(g) * u, else the plain product
    const void* rows;       // bf16 [max_rows][red]
    const void* w;
    const int32_t* offsets; // [E+1], device
    int32_t E;
    int64_t max_rows;       // 1 .. INT32_MAX
    int32_t red;            // multiple of 8 (mxfp4: of 32)
    int32_t feats;          // features of the output, multiple of 8 (mxfp4 gated: of 16)
    int32_t activation;
    void* out;              // bf16 [max_rows][feats]
    float* pre;             // gated: [max_rows][2 feats] or null
    int32_t zero;           // as above
};
// Whether a forward product is streamed, by a rule on the sizes; `positions`
// are rows of weights (two per feature if gated).
bool expert_streams_bf16(int64_t max_rows);
bool expert_streams_mxfp4(int32_t E, int64_t max_rows, int64_t positions);
hipError_t launch_expert_stream(const ExpertStreamArgs& a, hipStream_t stream);
int64_t expert_stream_grid(const ExpertStreamArgs& a);
// The same products with packed 4-bit weights for many rows per expert.
hipError_t launch_expert_mxfp4(const ExpertStreamArgs& a, hipStream_t stream);
int64_t expert_mxfp4_grid(const ExpertStreamArgs& a);

}  // namespace moe
