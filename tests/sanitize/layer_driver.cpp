// Drives every entry point of layer_api.cpp with valid and invalid arguments,
// the largest sizes among them, and counts what would have been launched.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "moe.h"

namespace moe {
extern int g_route, g_route_grad, g_quant, g_dequant, g_mx4, g_mx4_stream, g_layer;
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
    char* b[9];
    for (int i = 1; i < 9; ++i) b[i] = reinterpret_cast<char*>(uintptr_t(i) << 56);
    auto* i1 = reinterpret_cast<int32_t*>(b[5]);
    auto* f1 = reinterpret_cast<float*>(b[6]);
    auto* f2 = reinterpret_cast<float*>(b[7]);
    const int32_t tokens[] = {1, 64, 4097, (1 << 26) - 1};
    for (int32_t T : tokens) {
        EXPECT(moe_route_topk(b[1], MOE_F32, f2, T, 1024, 16, MOE_SCORE_SIGMOID, 1, 2.5f, 64, 64,
                              i1, f1, nullptr) == MOE_OK);
        EXPECT(moe_route_topk(b[1], MOE_BF16, nullptr, T, 1, 1, MOE_SCORE_SOFTMAX, 0, 1.0f, 1, 1,
                              i1, f1, nullptr) == MOE_OK);
        EXPECT(moe_route_topk_backward(b[1], MOE_BF16, i1, f1, T, 1024, 16, MOE_SCORE_SOFTMAX, 0,
                                       1.0f, b[2], nullptr) == MOE_OK);
    }
    EXPECT(moe::g_route == 8 && moe::g_route_grad == 4);
    EXPECT(moe_route_topk(b[1], MOE_F32, nullptr, 1 << 26, 8, 2, 0, 0, 1.0f, 1, 1, i1, f1,
                          nullptr) != MOE_OK);
    EXPECT(moe_route_topk(b[1], MOE_F32, nullptr, 4, 8, 2, 0, 0, NAN, 1, 1, i1, f1, nullptr) !=
           MOE_OK);
    EXPECT(moe_route_topk(b[1], MOE_F32, nullptr, 4, 8, 2, 0, 0, 1.0f, 0, 1, i1, f1, nullptr) !=
           MOE_OK);
    EXPECT(moe_route_topk(b[1], MOE_F32, nullptr, 4, 8, 2, 0, 0, 1.0f, INT32_MIN, 1, i1, f1,
                          nullptr) != MOE_OK);
    EXPECT(moe_route_topk(b[1], MOE_F32, nullptr, INT32_MIN, 8, 2, 0, 0, 1.0f, 1, 1, i1, f1,
                          nullptr) != MOE_OK);
    EXPECT(moe::g_route == 8);

    const int64_t rows[] = {1, 613, (int64_t(1) << 30) - 64, INT64_MAX};
    for (int64_t r : rows)
        for (int32_t width : {32, 7168, MOE_MAX_GEMM_WIDTH, INT32_MAX}) {
            const bool ok = width <= MOE_MAX_GEMM_WIDTH &&
                            r <= ((int64_t(1) << 30) - 64) / (width / 32);
            EXPECT((moe_quantize_mxfp4(b[1], MOE_BF16, r, width, b[2], b[3], nullptr) == MOE_OK) ==
                   ok);
            EXPECT((moe_dequantize_mxfp4(b[2], b[3], MOE_F32, r, width, b[1], nullptr) == MOE_OK) ==
                   ok);
        }
    EXPECT(moe::g_quant > 0 && moe::g_quant == moe::g_dequant);

    for (int64_t r : {int64_t(1), int64_t(64), int64_t(32768), int64_t(INT32_MAX)})
        for (int32_t E : {1, 256, MOE_MAX_EXPERTS}) {
            EXPECT(moe_grouped_gemm_mxfp4_rows(b[1], b[2], b[3], i1, E, r, 2880, 200, b[6], 9,
                                               nullptr) == MOE_OK);
            EXPECT(moe_gated_grouped_gemm_mxfp4_rows(b[1], b[2], b[3], i1, E, r, 7168, 2048,
                                                     MOE_ACT_GELU_TANH, b[6], 0, nullptr) ==
                   MOE_OK);
        }
    EXPECT(moe::g_mx4 > 0 && moe::g_mx4_stream > 0);
    EXPECT(moe_gated_grouped_gemm_mxfp4_rows(b[1], b[2], b[3], i1, 1, 8, 64, INT32_MAX, 0, b[6], 0,
                                             nullptr) != MOE_OK);
    EXPECT(moe_grouped_gemm_mxfp4_rows(b[1], b[2], b[3], i1, MOE_MAX_EXPERTS, 8, MOE_MAX_GEMM_WIDTH,
                                       MOE_MAX_GEMM_WIDTH, b[6], 0, nullptr) != MOE_OK);

    for (int32_t K : {1, 7, 16})
        for (int32_t layout : {MOE_WEIGHTS_ROW_MAJOR, MOE_WEIGHTS_MXFP4}) {
            const int32_t T = MOE_MAX_LAYER_SLOTS / K;
            const int64_t need = moe_few_tokens_workspace_bytes(T, K, 2048);
            EXPECT(need == int64_t(T) * K * 2048 * 4);
            EXPECT(moe_few_tokens_layer(b[1], f1, i1, T, K, b[2], b[3], layout, 256, 7168, 2048, 0,
                                        b[4], need, b[8], nullptr) == MOE_OK);
            EXPECT(moe_few_tokens_layer(b[1], f1, i1, T + 1, K, b[2], b[3], layout, 256, 7168, 2048,
                                        0, b[4], need * 2, b[8], nullptr) != MOE_OK);
            EXPECT(moe_few_tokens_layer(b[1], f1, i1, T, K, b[2], b[3], layout, 256, 7168, 2048, 0,
                                        b[4], need - 1, b[8], nullptr) == MOE_ERR_WORKSPACE);
        }
    EXPECT(moe::g_layer == 6);
    EXPECT(moe_few_tokens_workspace_bytes(INT32_MAX, 16, 2048) == -1);
    EXPECT(moe_few_tokens_workspace_bytes(1, INT32_MAX, 2048) == -1);
    EXPECT(moe_few_tokens_layer(b[1], f1, i1, 1, 1, b[2], b[3], MOE_WEIGHTS_ROW_MAJOR, 1024,
                                MOE_MAX_GEMM_WIDTH, MOE_MAX_GEMM_WIDTH / 2, 0, b[4],
                                int64_t(1) << 40, b[8], nullptr) == MOE_OK);
    EXPECT(moe::g_layer == 7);
    std::printf("%d failures\n", failures);
    return failures != 0;
}
