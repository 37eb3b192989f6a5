// Drives every entry point of the expert feed-forward block (expert_api.cpp)
// with valid and invalid arguments and counts what would have been launched.
#include <cstdint>
#include <cstdio>

#include "moe.h"

namespace moe {
extern int g_gemm, g_wgrad, g_stream, g_mxfp4, g_pack;
}

static int failures = 0;
#define EXPECT(c)                                                       \
    do {                                                                \
        if (!(c)) {                                                     \
            std::printf("line %d: %s\n", __LINE__, #c);                 \
            ++failures;                                                 \
        }                                                               \
    } while (0)

int main() {
    // Buffers that are never dereferenced, 2^56 bytes apart.
    char* p = reinterpret_cast<char*>(uintptr_t(1) << 56);
    char* w = p + (uintptr_t(1) << 56);
    char* out = w + (uintptr_t(1) << 56);
    auto* off = reinterpret_cast<const int32_t*>(out + (uintptr_t(1) << 56));
    auto* f32 = reinterpret_cast<float*>(out + (uintptr_t(2) << 56));
    const int32_t experts[] = {1, 256, MOE_MAX_EXPERTS};
    const int64_t sizes[] = {1, 64, 65, 2048, 32768, INT32_MAX};
    for (int64_t rows : sizes)
        for (int32_t E : experts) {
            EXPECT(moe_gated_grouped_gemm(p, w, off, E, rows, 7168, 2048, MOE_ACT_SILU, out, f32,
                                          MOE_GEMM_ZERO_TAIL, nullptr) == MOE_OK || rows == INT32_MAX);
            EXPECT(moe_grouped_gemm_forward(p, w, off, E, rows, 72, 200, out, 0, nullptr) == MOE_OK ||
                   rows == INT32_MAX);
            EXPECT(moe_grouped_gemm_backward_input(p, w, off, E, rows, 72, 200, out, 0, nullptr) ==
                       MOE_OK || rows == INT32_MAX);
            EXPECT(moe_gated_grouped_gemm_backward(p, w, f32, off, E, rows, 72, 200,
                                                   MOE_ACT_GELU_TANH, out, 0, nullptr) == MOE_OK ||
                   rows == INT32_MAX);
            EXPECT(moe_grouped_gemm_backward_weight(p, w, off, E, rows, 72, 200, MOE_F32, out,
                                                    MOE_GEMM_ACCUMULATE, nullptr) == MOE_OK);
            EXPECT(moe_grouped_gemm_mxfp4(p, w, off, E, rows, 2880, 200, out, 0, nullptr) == MOE_OK ||
                   rows == INT32_MAX);
            EXPECT(moe_gated_grouped_gemm_mxfp4(p, w, off, E, rows, 2880, 208, MOE_ACT_SILU, out, 0,
                                                nullptr) == MOE_OK || rows == INT32_MAX);
        }
    EXPECT(moe::g_gemm > 0 && moe::g_wgrad > 0 && moe::g_stream > 0 && moe::g_mxfp4 > 0);
    const int before = moe::g_gemm + moe::g_wgrad + moe::g_stream + moe::g_mxfp4;
    EXPECT(moe_gated_grouped_gemm(p, w, off, 1, 8, 7166, 2048, 0, out, nullptr, 0, nullptr) != MOE_OK);
    EXPECT(moe_gated_grouped_gemm(p, w, off, 1, 8, 64, 64, 7, out, nullptr, 0, nullptr) != MOE_OK);
    EXPECT(moe_gated_grouped_gemm(p + 8, w, off, 1, 8, 64, 64, 0, out, nullptr, 0, nullptr) != MOE_OK);
    EXPECT(moe_grouped_gemm_forward(nullptr, w, off, 1, 8, 64, 64, out, 0, nullptr) != MOE_OK);
    EXPECT(moe_grouped_gemm_forward(p, w, off, 1, 8, 64, 64, out, 2, nullptr) != MOE_OK);
    EXPECT(moe_grouped_gemm_forward(p, w, off, 1, 0, 64, 64, out, 0, nullptr) == MOE_OK);
    EXPECT(moe_grouped_gemm_backward_input(p, w, nullptr, 1, 8, 64, 64, out, 0, nullptr) != MOE_OK);
    EXPECT(moe_gated_grouped_gemm_backward(p, w, nullptr, off, 1, 8, 64, 64, 0, out, 0, nullptr) !=
           MOE_OK);
    EXPECT(moe_grouped_gemm_backward_weight(p, w, off, 1, 8, 64, 64, 9, out, 0, nullptr) != MOE_OK);
    EXPECT(moe_grouped_gemm_backward_weight(p, w, off, 1, 8, 64, 64, 0, nullptr, 0, nullptr) !=
           MOE_OK);
    EXPECT(moe_grouped_gemm_mxfp4(p, w, off, 1, 8, 48, 64, out, 0, nullptr) != MOE_OK);
    EXPECT(moe_gated_grouped_gemm_mxfp4(p, w, off, 1, 8, 64, 24, 0, out, 0, nullptr) != MOE_OK);
    // Outputs that touch an input, and one that ends where the inputs begin.
    EXPECT(moe_grouped_gemm_forward(p, w, off, 1, 8, 64, 64, p + 1008, 0, nullptr) != MOE_OK);
    EXPECT(moe_grouped_gemm_forward(p, w, off, 1, 8, 64, 64, w - 1008, 0, nullptr) != MOE_OK);
    EXPECT(moe_gated_grouped_gemm(p, w, off, 1, 8, 64, 64, 0, out,
                                  reinterpret_cast<float*>(out + 1008), 0, nullptr) != MOE_OK);
    EXPECT(before == moe::g_gemm + moe::g_wgrad + moe::g_stream + moe::g_mxfp4);
    EXPECT(moe_grouped_gemm_forward(p, w, off, 1, 8, 64, 64, p + 1024, 0, nullptr) == MOE_OK);
    EXPECT(moe_grouped_gemm_forward(p, w, off, 1, 8, 64, 64, w - 1024, 0, nullptr) == MOE_OK);
    // Without rows nothing is read, so nothing can be shared.
    EXPECT(moe_grouped_gemm_backward_weight(out + 64, out + 64, off, 1, 0, 64, 64, MOE_F32, out, 0,
                                            nullptr) == MOE_OK);
    EXPECT(moe_mxfp4_weights_bytes(2, 24, 160) == 2 * 2 * 2 * 1088);
    EXPECT(moe_mxfp4_weights_bytes(MOE_MAX_EXPERTS, MOE_MAX_GEMM_WIDTH, MOE_MAX_GEMM_WIDTH) == -1);
    EXPECT(moe_pack_mxfp4_weights(p, w, 2, 24, 160, out, nullptr) == MOE_OK && moe::g_pack == 1);
    EXPECT(moe_pack_mxfp4_weights(p + 4, w, 2, 24, 160, out, nullptr) != MOE_OK && moe::g_pack == 1);
    std::printf("%d failures\n", failures);
    return failures != 0;
}
