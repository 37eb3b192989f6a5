// Row counts up to the largest one a call takes, divided into tiles and steps
// as the kernels of the expert feed-forward block divide them.
#include <cstdint>
#include <cstdio>

#include "expert_kernels.h"

int main() {
    int failures = 0;
    for (int32_t size : {16, 32, 64, 256})
        for (int64_t rows : {int64_t(0), int64_t(1), int64_t(size), int64_t(size) + 1,
                             int64_t(INT32_MAX) - size, int64_t(INT32_MAX) - size + 2,
                             int64_t(INT32_MAX)}) {
            const int64_t want = (rows + size - 1) / size;
            const int64_t got = moe::expert_row_parts(static_cast<int32_t>(rows), size);
            if (got != want) {
                std::printf("%lld rows in parts of %d: %lld\n", static_cast<long long>(rows), size,
                            static_cast<long long>(got));
                ++failures;
            }
        }
    std::printf("%d failures\n", failures);
    return failures != 0;
}
