// MXFP4 on gfx950: rows to 4 bits and back. With top the largest magnitude of
// a block of 32 elements and e = max(floor(log2(top)) - 2, -127), an element x
// becomes the e2m1 number nearest to x / 2^e (ties to the even one; 6 is the
// largest, which what lies above it becomes too) and the block's scale byte
// e + 127. A block of zeros has byte 0, one with a NaN or an infinity 255, which
// makes all its elements NaN. x / 2^e is exact but where it falls below 2^-126,
// far under the smallest e2m1 number: one rounding in all.
//
// Bound: the bytes. Four lanes share a block, eight elements each, so that a lane's
// loads and stores are 16 or 32 bytes of the rows and 4 of the values, and the scale
// needs two exchanges within the four. Measured on MI355X: 32768 rows of 7168 in bf16,
// 595 MB, 116 us there and 104 us back (5.1 and 5.7 TB/s, a large copy 4.7); 613 rows of
// 1984 in fp32 2.3 and 3.2 us, a launch's time.
#include "expert_mma.h"
#include "layer_kernels.h"

namespace moe {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

struct Eight {
    float v[8];
};

__device__ __forceinline__ Eight load_eight(const float* p) {
    Eight r;
    const f32x4 a = *reinterpret_cast<const f32x4*>(p);
    const f32x4 b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.v[i] = a[i];
        r.v[4 + i] = b[i];
    }
    return r;
}
__device__ __forceinline__ Eight load_eight(const __bf16* p) {
    Eight r;
    const v4i a = *reinterpret_cast<const v4i*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.v[2 * i] = __uint_as_float(static_cast<uint32_t>(a[i]) << 16);
        r.v[2 * i + 1] = __uint_as_float(static_cast<uint32_t>(a[i]) & 0xFFFF0000u);
    }
    return r;
}

// The largest of a block's four lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true)));
    return max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true)));
}

template <class T>
__global__ __launch_bounds__(256)
void quantize_mxfp4_kernel(const T* __restrict__ src, int64_t blocks, uint32_t* __restrict__ values,
                           uint8_t* __restrict__ scales) {
    // Whole quads stay or leave together.
    const int64_t q = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (q >= blocks * 4) return;
    const Eight x = load_eight(src + q * 8);
    // Magnitudes compare as their bits; NaN lies above infinity.
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x.v[i]) & 0x7FFFFFFFu);
    top = quad_max(top);
    // floor(log2(top)) is the exponent field of a normal number; smaller ones
    // have e = -127 whatever it is, as have all below 2^-125.
    const int32_t field = static_cast<int32_t>(top >> 23);
    const bool lost = field == 255;
    const int32_t e = max(field - 127 - 2, -127);
    uint32_t word = 0;
    if (!lost) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = __builtin_amdgcn_ldexpf(x.v[i], -e);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, t[0], t[1], 1.0f, 0);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, t[2], t[3], 1.0f, 1);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, t[4], t[5], 1.0f, 2);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, t[6], t[7], 1.0f, 3);
    }
    values[q] = word;
    if ((threadIdx.x & 3) == 0) scales[q >> 2] = static_cast<uint8_t>(lost ? 255 : e + 127);
}

__device__ __forceinline__ void store_eight(float* p, const float (&v)[8]) {
    *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store_eight(__bf16* p, const float (&v)[8]) {
    const v2i a = pack_bf16x4(f32x4{v[0], v[1], v[2], v[3]});
    const v2i b = pack_bf16x4(f32x4{v[4], v[5], v[6], v[7]});
    *reinterpret_cast<v4i*>(p) = v4i{a[0], a[1], b[0], b[1]};
}

template <class T>
__global__ __launch_bounds__(256)
void dequantize_mxfp4_kernel(const uint32_t* __restrict__ values,
                             const uint8_t* __restrict__ scales, int64_t blocks,
                             T* __restrict__ dst) {
    const int64_t q = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (q >= blocks * 4) return;
    const uint32_t w = values[q];
    const int32_t s = scales[q >> 2];
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto p = i == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0)
                       : i == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1)
                       : i == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2)
                                : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
        v[2 * i] = __builtin_amdgcn_ldexpf(p[0], s - 127);
        v[2 * i + 1] = __builtin_amdgcn_ldexpf(p[1], s - 127);
    }
    if (s == 255) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(0x7FC00000u);
    }
    store_eight(dst + q * 8, v);
}

dim3 quant_grid(int64_t blocks) { return dim3(static_cast<uint32_t>((blocks * 4 + 255) / 256)); }

}  // namespace

hipError_t launch_quantize_mxfp4(const QuantArgs& a, hipStream_t stream) {
    if (a.bf16)
        hipLaunchKernelGGL((quantize_mxfp4_kernel<__bf16>), quant_grid(a.blocks), dim3(256), 0,
                           stream, static_cast<const __bf16*>(a.src), a.blocks,
                           static_cast<uint32_t*>(a.values), a.scales);
    else
        hipLaunchKernelGGL((quantize_mxfp4_kernel<float>), quant_grid(a.blocks), dim3(256), 0,
                           stream, static_cast<const float*>(a.src), a.blocks,
                           static_cast<uint32_t*>(a.values), a.scales);
    return hipGetLastError();
}

hipError_t launch_dequantize_mxfp4(const QuantArgs& a, hipStream_t stream) {
    if (a.bf16)
        hipLaunchKernelGGL((dequantize_mxfp4_kernel<__bf16>), quant_grid(a.blocks), dim3(256), 0,
                           stream, static_cast<const uint32_t*>(a.values), a.scales, a.blocks,
                           static_cast<__bf16*>(a.dst));
    else
        hipLaunchKernelGGL((dequantize_mxfp4_kernel<float>), quant_grid(a.blocks), dim3(256), 0,
                           stream, static_cast<const uint32_t*>(a.values), a.scales, a.blocks,
                           static_cast<float*>(a.dst));
    return hipGetLastError();
}

}  // namespace moe
