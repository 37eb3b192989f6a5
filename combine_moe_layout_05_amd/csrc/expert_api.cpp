// C ABI entry points of the expert feed-forward block (include/moe.h): host
// argument checks and the choice of kernel. No entry point touches the device
// before every check has passed.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>
#include <initializer_list>

#include "expert_kernels.h"
#include "moe.h"

namespace moe {

// Where the form that streams the weights (16-row tiles, the sum split over a
// workgroup's wavefronts) is the faster one. Measured on MI355X with other
// weights in every call, so that they come from HBM, streamed against tiled:
//   - bf16, up to 64 rows: one expert of 4096 -> 2 x 2048 gated 19.7 and 31.4 us
//     at 32 rows, 19.7 and 32.9 at 64, 33.9 and 30.2 at 65, 64.0 and 31.9 at 256;
//     one of 2048 -> 7168 13.3 and 18.1 at 32 rows, 19.9 and 19.1 at 64, 26.8 and
//     17.8 at 65. With more experts they come near, on either side: at 64 rows 64
//     of 7168 -> 2 x 2048 623 and 626, 8 of 4096 -> 2 x 2048 58.6 and 51.1.
//   - 4 bits, up to 8 rows per expert: 128 experts of 4096 -> 2 x 2048 182 and 199
//     us at 1024 rows, 203 and 202 at 2048.
//   - 4 bits, while its workgroups are few (the tiled form then leaves CUs
//     idle): one expert of 4096 -> 2 x 2048 20.3 and 40.2 us at 256 rows (1024
//     workgroups), 39.0 and 40.6 at 512 (2048); 8 of 4096 -> 2 x 1408 31.5 and 42.9
//     at 512 (1408), 48.6 and 39.9 at 768 (2112); one of 2048 -> 7168 21.2 and 23.0
//     at 256 (1792), 38.2 and 23.8 at 512 (3584).
bool expert_streams_bf16(int64_t max_rows) { return max_rows <= 64; }
bool expert_streams_mxfp4(int32_t E, int64_t max_rows, int64_t positions) {
    if (max_rows <= int64_t(8) * E) return true;
    const int64_t experts = max_rows < E ? max_rows : E;
    const int64_t tiles = (max_rows + 15) / 16;
    return (positions + 63) / 64 * (tiles > experts ? tiles : experts) <= 1536;
}

}  // namespace moe

namespace {

bool misaligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0;
}

bool width_ok(int32_t n, int32_t multiple) {
    return n >= 8 && n <= MOE_MAX_GEMM_WIDTH && n % multiple == 0;
}

bool experts_ok(int32_t E) { return E >= 1 && E <= MOE_MAX_EXPERTS; }

bool activation_ok(int32_t a) { return a == MOE_ACT_SILU || a == MOE_ACT_GELU_TANH; }

// Whether two buffers share a byte. The sizes stay below 2^56 bytes.
bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    if (a_bytes == 0 || b_bytes == 0) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return pa < pb ? pb - pa < static_cast<uintptr_t>(a_bytes)
                   : pa - pb < static_cast<uintptr_t>(b_bytes);
}

// A buffer a call reads.
struct Input {
    const void* p;
    int64_t bytes;
};
Input rows_of(const void* p, int64_t rows, int64_t width, int64_t elem = 2) {
    return {p, rows * width * elem};
}
Input weights_of(const void* p, int64_t E, int64_t n, int64_t k) { return {p, E * n * k * 2}; }
Input offsets_of(const int32_t* p, int32_t E) { return {p, (int64_t(E) + 1) * 4}; }

// An output that shares bytes with none of the inputs: other workgroups still
// read those when it is written.
bool apart(const void* out, int64_t bytes, std::initializer_list<Input> inputs) {
    for (const Input& in : inputs)
        if (overlap(out, bytes, in.p, in.bytes)) return false;
    return true;
}

// bf16 buffers every call of the family needs, with its offsets.
bool buffers_ok(const void* a, const void* b, const void* c, const int32_t* offsets) {
    return a && b && c && offsets && !misaligned(a, 16) && !misaligned(b, 16) &&
           !misaligned(c, 16) && !misaligned(offsets, 4);
}

constexpr int32_t kZeroFlags = MOE_GEMM_ZERO_TAIL | MOE_GEMM_ZERO_HEAD;
int32_t zero_of(int32_t flags) {
    return ((flags & MOE_GEMM_ZERO_TAIL) ? moe::kZeroTail : 0) |
           ((flags & MOE_GEMM_ZERO_HEAD) ? moe::kZeroHead : 0);
}

int status_of(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

int run_gemm(moe::ExpertOp op, const void* rows, const void* w, const int32_t* offsets, int32_t E,
             int64_t max_rows, int32_t red, int32_t feats, int32_t activation, void* out,
             float* pre, int32_t flags, void* stream) {
    const bool forward = op == moe::ExpertOp::kPlain || op == moe::ExpertOp::kGated;
    if (forward && moe::expert_streams_bf16(max_rows)) {
        moe::ExpertStreamArgs a;
        a.mxfp4 = false;
        a.gated = op == moe::ExpertOp::kGated;
        a.rows = rows;
        a.w = w;
        a.offsets = offsets;
        a.E = E;
        a.max_rows = max_rows;
        a.red = red;
        a.feats = feats;
        a.activation = activation;
        a.out = out;
        a.pre = pre;
        a.zero = zero_of(flags);
        if (moe::expert_stream_grid(a) > moe::kMaxGrid) return MOE_ERR_INVALID_ARG;
        return status_of(moe::launch_expert_stream(a, static_cast<hipStream_t>(stream)));
    }
    moe::ExpertGemmArgs a;
    a.op = op;
    a.rows = rows;
    a.w = w;
    a.offsets = offsets;
    a.E = E;
    a.max_rows = max_rows;
    a.red = red;
    a.feats = feats;
    a.activation = activation;
    a.out = out;
    a.pre = pre;
    a.zero = zero_of(flags);
    if (moe::expert_gemm_grid(a) > moe::kMaxGrid) return MOE_ERR_INVALID_ARG;
    return status_of(moe::launch_expert_gemm(a, static_cast<hipStream_t>(stream)));
}

int run_mxfp4(bool gated, const void* rows, const void* packed, const int32_t* offsets, int32_t E,
              int64_t max_rows, int32_t red, int32_t feats, int32_t activation, void* out,
              int32_t flags, void* stream) {
    const int64_t packed_bytes = moe_mxfp4_weights_bytes(E, gated ? 2 * feats : feats, red);
    if (packed_bytes < 0) return MOE_ERR_INVALID_ARG;
    if (max_rows < 0 || max_rows > INT32_MAX || (flags & ~kZeroFlags))
        return MOE_ERR_INVALID_ARG;
    if (max_rows == 0) return MOE_OK;
    if (!buffers_ok(rows, packed, out, offsets) ||
        !apart(out, max_rows * feats * 2,
               {rows_of(rows, max_rows, red), {packed, packed_bytes}, offsets_of(offsets, E)}))
        return MOE_ERR_INVALID_ARG;
    moe::ExpertStreamArgs a;
    a.mxfp4 = true;
    a.gated = gated;
    a.rows = rows;
    a.w = packed;
    a.offsets = offsets;
    a.E = E;
    a.max_rows = max_rows;
    a.red = red;
    a.feats = feats;
    a.activation = activation;
    a.out = out;
    a.pre = nullptr;
    a.zero = zero_of(flags);
    if (moe::expert_streams_mxfp4(E, max_rows, gated ? int64_t(2) * feats : feats)) {
        if (moe::expert_stream_grid(a) > moe::kMaxGrid) return MOE_ERR_INVALID_ARG;
        return status_of(moe::launch_expert_stream(a, static_cast<hipStream_t>(stream)));
    }
    if (moe::expert_mxfp4_grid(a) > moe::kMaxGrid) return MOE_ERR_INVALID_ARG;
    return status_of(moe::launch_expert_mxfp4(a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int moe_gated_grouped_gemm(const void* d_x_expert, const void* d_weights,
                           const int32_t* d_offsets, int32_t num_experts, int64_t max_rows,
                           int32_t k_in, int32_t n_hidden, int32_t activation, void* d_h,
                           float* d_pre, int32_t flags, void* stream) {
    if (!experts_ok(num_experts) || !width_ok(k_in, 8) || !width_ok(n_hidden, 8) ||
        !activation_ok(activation) || max_rows < 0 || max_rows > INT32_MAX ||
        (flags & ~kZeroFlags))
        return MOE_ERR_INVALID_ARG;
    if (max_rows == 0) return MOE_OK;
    if (!buffers_ok(d_x_expert, d_weights, d_h, d_offsets) || (d_pre && misaligned(d_pre, 16)))
        return MOE_ERR_INVALID_ARG;
    const Input x = rows_of(d_x_expert, max_rows, k_in);
    const Input w = weights_of(d_weights, num_experts, int64_t(2) * n_hidden, k_in);
    const Input off = offsets_of(d_offsets, num_experts);
    const Input h = rows_of(d_h, max_rows, n_hidden);
    if (!apart(d_h, h.bytes, {x, w, off}) ||
        (d_pre && !apart(d_pre, max_rows * n_hidden * 8, {x, w, off, h})))
        return MOE_ERR_INVALID_ARG;
    return run_gemm(moe::ExpertOp::kGated, d_x_expert, d_weights, d_offsets, num_experts, max_rows,
                    k_in, n_hidden, activation, d_h, d_pre, flags, stream);
}

int moe_grouped_gemm_forward(const void* d_x_expert, const void* d_weights,
                             const int32_t* d_offsets, int32_t num_experts, int64_t max_rows,
                             int32_t k_in, int32_t n_out, void* d_out, int32_t flags,
                             void* stream) {
    if (!experts_ok(num_experts) || !width_ok(k_in, 8) || !width_ok(n_out, 8) || max_rows < 0 ||
        max_rows > INT32_MAX || (flags & ~kZeroFlags))
        return MOE_ERR_INVALID_ARG;
    if (max_rows == 0) return MOE_OK;
    if (!buffers_ok(d_x_expert, d_weights, d_out, d_offsets) ||
        !apart(d_out, max_rows * n_out * 2,
               {rows_of(d_x_expert, max_rows, k_in),
                weights_of(d_weights, num_experts, n_out, k_in),
                offsets_of(d_offsets, num_experts)}))
        return MOE_ERR_INVALID_ARG;
    return run_gemm(moe::ExpertOp::kPlain, d_x_expert, d_weights, d_offsets, num_experts, max_rows,
                    k_in, n_out, MOE_ACT_SILU, d_out, nullptr, flags, stream);
}

int moe_grouped_gemm_backward_input(const void* d_grad_out, const void* d_weights,
                                    const int32_t* d_offsets, int32_t num_experts,
                                    int64_t max_rows, int32_t k_in, int32_t n_out,
                                    void* d_grad_x, int32_t flags, void* stream) {
    if (!experts_ok(num_experts) || !width_ok(k_in, 8) || !width_ok(n_out, 8) || max_rows < 0 ||
        max_rows > INT32_MAX || (flags & ~kZeroFlags))
        return MOE_ERR_INVALID_ARG;
    if (max_rows == 0) return MOE_OK;
    if (!buffers_ok(d_grad_out, d_weights, d_grad_x, d_offsets) ||
        !apart(d_grad_x, max_rows * k_in * 2,
               {rows_of(d_grad_out, max_rows, n_out),
                weights_of(d_weights, num_experts, n_out, k_in),
                offsets_of(d_offsets, num_experts)}))
        return MOE_ERR_INVALID_ARG;
    return run_gemm(moe::ExpertOp::kInputGrad, d_grad_out, d_weights, d_offsets, num_experts,
                    max_rows, n_out, k_in, MOE_ACT_SILU, d_grad_x, nullptr, flags, stream);
}

int moe_gated_grouped_gemm_backward(const void* d_grad_out, const void* d_weights,
                                    const float* d_pre, const int32_t* d_offsets,
                                    int32_t num_experts, int64_t max_rows, int32_t n_hidden,
                                    int32_t n_out, int32_t activation, void* d_grad_pre,
                                    int32_t flags, void* stream) {
    if (!experts_ok(num_experts) || !width_ok(n_hidden, 8) || !width_ok(n_out, 8) ||
        !activation_ok(activation) || max_rows < 0 || max_rows > INT32_MAX ||
        (flags & ~kZeroFlags))
        return MOE_ERR_INVALID_ARG;
    if (max_rows == 0) return MOE_OK;
    if (!buffers_ok(d_grad_out, d_weights, d_grad_pre, d_offsets) || !d_pre ||
        misaligned(d_pre, 16) ||
        !apart(d_grad_pre, max_rows * n_hidden * 4,
               {rows_of(d_grad_out, max_rows, n_out),
                weights_of(d_weights, num_experts, n_out, n_hidden),
                rows_of(d_pre, max_rows, int64_t(2) * n_hidden, 4),
                offsets_of(d_offsets, num_experts)}))
        return MOE_ERR_INVALID_ARG;
    return run_gemm(moe::ExpertOp::kGatedGrad, d_grad_out, d_weights, d_offsets, num_experts,
                    max_rows, n_out, n_hidden, activation, d_grad_pre,
                    const_cast<float*>(d_pre), flags, stream);
}

int moe_grouped_gemm_backward_weight(const void* d_grad_out, const void* d_x_expert,
                                     const int32_t* d_offsets, int32_t num_experts,
                                     int64_t max_rows, int32_t k_in, int32_t n_out,
                                     int32_t grad_dtype, void* d_grad_w, int32_t flags,
                                     void* stream) {
    if (!experts_ok(num_experts) || !width_ok(k_in, 8) || !width_ok(n_out, 8) || max_rows < 0 ||
        max_rows > INT32_MAX || (grad_dtype != MOE_BF16 && grad_dtype != MOE_F32) ||
        (flags & ~MOE_GEMM_ACCUMULATE))
        return MOE_ERR_INVALID_ARG;
    if (!d_grad_w || !d_offsets || misaligned(d_grad_w, 16) || misaligned(d_offsets, 4))
        return MOE_ERR_INVALID_ARG;
    // Without rows nothing is read: the gradient is zero (or stays).
    if (max_rows > 0 && (!d_grad_out || !d_x_expert || misaligned(d_grad_out, 16) ||
                         misaligned(d_x_expert, 16)))
        return MOE_ERR_INVALID_ARG;
    if (!apart(d_grad_w,
               int64_t(num_experts) * n_out * k_in * (grad_dtype == MOE_F32 ? 4 : 2),
               {rows_of(d_grad_out, max_rows, n_out), rows_of(d_x_expert, max_rows, k_in),
                offsets_of(d_offsets, num_experts)}))
        return MOE_ERR_INVALID_ARG;
    moe::ExpertWgradArgs a;
    a.dy = d_grad_out;
    a.x = d_x_expert;
    a.offsets = d_offsets;
    a.E = num_experts;
    a.max_rows = max_rows;
    a.N = n_out;
    a.K = k_in;
    a.f32 = grad_dtype == MOE_F32;
    a.accumulate = (flags & MOE_GEMM_ACCUMULATE) != 0;
    a.dw = d_grad_w;
    if (moe::expert_wgrad_grid(a) > moe::kMaxGrid) return MOE_ERR_INVALID_ARG;
    return status_of(moe::launch_expert_wgrad(a, static_cast<hipStream_t>(stream)));
}

int64_t moe_mxfp4_weights_bytes(int32_t num_experts, int32_t n_out, int32_t k_in) {
    if (!experts_ok(num_experts) || !width_ok(n_out, 8) || !width_ok(k_in, 32)) return -1;
    if (moe::mxfp4_pack_grid(num_experts, n_out, k_in) > moe::kMaxGrid) return -1;
    return moe::mxfp4_bytes(num_experts, n_out, k_in);
}

int moe_pack_mxfp4_weights(const void* d_values, const void* d_scales, int32_t num_experts,
                           int32_t n_out, int32_t k_in, void* d_packed, void* stream) {
    const int64_t bytes = moe_mxfp4_weights_bytes(num_experts, n_out, k_in);
    if (bytes < 0) return MOE_ERR_INVALID_ARG;
    if (!d_values || !d_scales || !d_packed || misaligned(d_values, 16) || misaligned(d_packed, 16))
        return MOE_ERR_INVALID_ARG;
    const int64_t values = int64_t(num_experts) * n_out * k_in;
    if (!apart(d_packed, bytes, {{d_values, values / 2}, {d_scales, values / 32}}))
        return MOE_ERR_INVALID_ARG;
    moe::PackMxfp4Args a;
    a.blocks = d_values;
    a.scales = d_scales;
    a.E = num_experts;
    a.N = n_out;
    a.K = k_in;
    a.dst = d_packed;
    return status_of(moe::launch_pack_mxfp4(a, static_cast<hipStream_t>(stream)));
}

int moe_grouped_gemm_mxfp4(const void* d_x_expert, const void* d_packed, const int32_t* d_offsets,
                           int32_t num_experts, int64_t max_rows, int32_t k_in, int32_t n_out,
                           void* d_out, int32_t flags, void* stream) {
    return run_mxfp4(false, d_x_expert, d_packed, d_offsets, num_experts, max_rows, k_in, n_out,
                     MOE_ACT_SILU, d_out, flags, stream);
}

int moe_gated_grouped_gemm_mxfp4(const void* d_x_expert, const void* d_packed,
                                 const int32_t* d_offsets, int32_t num_experts, int64_t max_rows,
                                 int32_t k_in, int32_t n_hidden, int32_t activation, void* d_h,
                                 int32_t flags, void* stream) {
    if (!width_ok(n_hidden, 16) || n_hidden > MOE_MAX_GEMM_WIDTH / 2 || !activation_ok(activation))
        return MOE_ERR_INVALID_ARG;
    return run_mxfp4(true, d_x_expert, d_packed, d_offsets, num_experts, max_rows, k_in, n_hidden,
                     activation, d_h, flags, stream);
}

}  // extern "C"
