// Argument checks that the C entry points of the expert products and of the
// layer around them share. Host code only.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "expert_kernels.h"
#include "moe.h"

namespace moe {

inline bool misaligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0;
}

inline bool width_ok(int32_t n, int32_t multiple) {
    return n >= 8 && n <= MOE_MAX_GEMM_WIDTH && n % multiple == 0;
}

inline bool experts_ok(int32_t E) { return E >= 1 && E <= MOE_MAX_EXPERTS; }

inline bool activation_ok(int32_t a) { return a == MOE_ACT_SILU || a == MOE_ACT_GELU_TANH; }

// Whether two buffers share a byte. The sizes stay below 2^56 bytes.
inline bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
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
inline Input rows_of(const void* p, int64_t rows, int64_t width, int64_t elem = 2) {
    return {p, rows * width * elem};
}
inline Input weights_of(const void* p, int64_t E, int64_t n, int64_t k) { return {p, E * n * k * 2}; }
inline Input offsets_of(const int32_t* p, int32_t E) { return {p, (int64_t(E) + 1) * 4}; }

// An output that shares bytes with none of the inputs: other workgroups still
// read those when it is written.
inline bool apart(const void* out, int64_t bytes, std::initializer_list<Input> inputs) {
    for (const Input& in : inputs)
        if (overlap(out, bytes, in.p, in.bytes)) return false;
    return true;
}

constexpr int32_t kZeroFlags = MOE_GEMM_ZERO_TAIL | MOE_GEMM_ZERO_HEAD;
inline int32_t zero_of(int32_t flags) {
    return ((flags & MOE_GEMM_ZERO_TAIL) ? kZeroTail : 0) |
           ((flags & MOE_GEMM_ZERO_HEAD) ? kZeroHead : 0);
}

inline int status_of(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace moe
