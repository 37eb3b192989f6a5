// Packed 4-bit weights in registers. Internal to libmoe_layout.so.
#pragma once

#include "expert_mma.h"

namespace moe {

// One 128-element step of a 16-feature block: this lane's 32 values and the
// scales of its feature's four groups of 32.
struct Mxfp4Step {
    v4i q;
    uint32_t scale;
    // The A fragment of the product over group s, as bf16: the conversion is
    // exact (2-bit significands times a power of two; the scale's byte is the
    // exponent field of a float, 255 giving NaN).
    __device__ bf16x8 frag(int s) const {
        const float f = __uint_as_float(((scale >> (8 * s)) & 0xFFu) << 23);
        const uint32_t v = static_cast<uint32_t>(q[s]);
        const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, f, 0);
        const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, f, 1);
        const auto c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, f, 2);
        const auto d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, f, 3);
        return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
};

}  // namespace moe
