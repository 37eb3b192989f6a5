// Expert products for few rows per expert on gfx950, and the packing of 4-bit
// expert weights: with rows r of expert e, out[r] = x[r] W^T, or act(g) * u of
// the two projections g and u.
//
// Bound: the bytes of the weights, each used for at most 16 rows; a segment's
// weights are read once per 16 of its rows. They go straight into the registers
// the matrix cores read, never through LDS: a workgroup takes 64 features, its
// wavefronts every n-th step of the sum (consecutive weights, so that a
// workgroup's reads are one stream), and the wavefronts' sums are joined in LDS
// in wavefront order. Splitting the sum gives one token enough workgroups and
// loads in flight: 8 experts' 4096 features are 512 workgroups of 8 wavefronts.
//
// Measured on MI355X, one token of 8 experts, other experts in every call, so that
// the weights come from HBM (a large copy moves 4.9 TB/s, an in-place update 6.0).
// bf16, 7168 -> 2 x 2048: 79.1 us for 470 MB (5.9 TB/s); 2048 -> 7168: 47.5 us for
// 235 MB (4.9). 4 bits, 7168 -> 2 x 2048: 22.4 us for 125 MB (5.6 TB/s); 2048 ->
// 7168: 14.2 us for 62 MB (4.4), where a wavefront has four steps and start and
// end weigh most. The same experts again, out of the memory-side cache: 78.7, 38.4,
// 20.4 and 12.7 us. 64 tokens over 256 experts at 4 bits: 330 to 350 us for 2.13 GB
// (6.1 to 6.5 TB/s).
#include "expert_kernels.h"
#include "expert_mma.h"
#include "expert_mxfp4.h"

#include <type_traits>

namespace moe {
namespace {

// Wavefronts of a workgroup, splitting the sum. 4-bit weights leave each little
// to read, and more, smaller workgroups start together: 14.2 against 16.5 us
// with 8 at one token of 2048 -> 7168 (8 experts, weights from HBM), 22.4 against
// 22.6 us at 7168 -> 2 x 2048. With bf16 weights 4 or 8 make no difference there
// (79.1 with 8, 78.9 with 4; 2048 -> 7168 47.5 and 46.7 us).
constexpr int waves_of(bool mxfp4) { return mxfp4 ? 4 : 8; }
constexpr int kBlocks = 4;              // 16-feature blocks per workgroup
constexpr int kRows = 16;               // rows per workgroup
constexpr int kXcdChunk = 32;

// Sum elements per step, the 32-element products in it and 16-byte chunks.
template <bool MXFP4>
struct Step {
    static constexpr int kElems = MXFP4 ? kMxfp4Step : 64;
    static constexpr int kProducts = kElems / 32;
    static constexpr int kRowChunks = kElems / 8;
    static constexpr int kRowLoads = kRows * kRowChunks / 64;
    static constexpr int kRowsPerLoad = 64 / kRowChunks;
};

// One step of a 16-feature block in registers.
template <bool MXFP4>
struct Weights;
template <>
struct Weights<true> : Mxfp4Step {};
template <>
struct Weights<false> {
    v4i q[2];
    __device__ bf16x8 frag(int s) const { return __builtin_bit_cast(bf16x8, q[s]); }
};

template <bool MXFP4, bool GATED>
__global__ __launch_bounds__(waves_of(MXFP4) * 64, 4)
void expert_stream_kernel(const char* __restrict__ rows, const char* __restrict__ w,
                          const char* __restrict__ scales, const int32_t* __restrict__ offsets,
                          int32_t E, int32_t max_rows, int32_t red, int32_t feats, int32_t ftiles,
                          int32_t act, char* __restrict__ out, float* __restrict__ pre,
                          int32_t zero) {
    typedef Step<MXFP4> S;
    constexpr int kWaves = waves_of(MXFP4);
    constexpr int kFeatBlocks = GATED ? kBlocks / 2 : kBlocks;  // of the output
    constexpr int kXs = kRows * S::kRowChunks;                  // chunks of a row step
    __shared__ v4i x0[kWaves][kXs], x1[kWaves][kXs];
    // The wavefronts' sums, [wave][block][lane]; with 4-bit weights they take
    // the place of the wavefront's own rows, so that two workgroups fit a CU.
    constexpr int kPart = kBlocks * 64;
    static_assert(!MXFP4 || kXs == kPart, "the sums fill the place of the rows");
    __shared__ v4i sums[MXFP4 ? 1 : kWaves][MXFP4 ? 1 : kPart];
    __shared__ int32_t info[4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t number = expert_tile_number(kXcdChunk);
    if (wave == 0) {
        // Feature tiles fastest: neighbouring workgroups read neighbouring
        // weights; the row tiles of a longer segment follow each other.
        const ExpertTile t = expert_find_tile(offsets, E, max_rows, kRows, ftiles, 4, number);
        if (lane == 0) {
            info[0] = t.e;
            info[1] = t.f;
            info[2] = t.row0;
            info[3] = t.rows;
        }
    }
    __syncthreads();
    const int32_t e = __builtin_amdgcn_readfirstlane(info[0]);
    const int32_t ft = __builtin_amdgcn_readfirstlane(info[1]);
    const int32_t row0 = __builtin_amdgcn_readfirstlane(info[2]);
    const int32_t nrows = __builtin_amdgcn_readfirstlane(info[3]);
    if (e < 0) {
        if (zero)
            expert_zero_rows(reinterpret_cast<v4i*>(out), offsets, zero, row0, max_rows, feats / 8,
                             ft, int64_t(gridDim.x) - nrows);
        return;
    }
    const int i = lane & 15, g = lane >> 4;
    const int32_t f0 = ft * kFeatBlocks * 16;
    const int32_t steps = (red + S::kElems - 1) / S::kElems;
    const int32_t full = red / S::kElems;

    // Weight addresses of the 16-feature blocks; blocks past the matrix read
    // its last one and are not stored.
    const char* wb[kBlocks];
    const char* sb[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        const int ob = GATED ? b % kFeatBlocks : b;         // output block
        const bool up = GATED && b >= kFeatBlocks;
        if constexpr (MXFP4) {
            const int32_t nb = (feats + 15) / 16;
            const int64_t blk = int64_t(e) * nb * (GATED ? 2 : 1) + (up ? nb : 0) +
                                min(f0 / 16 + ob, nb - 1);
            wb[b] = w + blk * steps * 1024 + lane * 16;
            sb[b] = scales + blk * steps * 64 + i * 4;
        } else {
            const int32_t f = min(f0 + ob * 16 + i, feats - 1) + (up ? feats : 0);
            wb[b] = w + (int64_t(e) * feats * (GATED ? 2 : 1) + f) * (int64_t(red) * 2) + g * 16;
            sb[b] = nullptr;
        }
    }
    const int64_t pitch = int64_t(red) * 2;
    auto load_w = [&](int32_t t, Weights<MXFP4> (&d)[kBlocks]) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            if constexpr (MXFP4) {
                d[b].q = __builtin_nontemporal_load(
                    reinterpret_cast<const v4i*>(wb[b] + int64_t(t) * 1024));
                d[b].scale = *reinterpret_cast<const uint32_t*>(sb[b] + int64_t(t) * 64);
            } else {
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    d[b].q[s] = *reinterpret_cast<const v4i*>(wb[b] + int64_t(t) * 128 + s * 64);
            }
        }
    };
    // Rows: chunk c of row r sits at chunk c ^ swizzle(r) of the row's step,
    // so that 16 rows at one chunk fall into distinct LDS banks.
    auto swz = [](int r) { return MXFP4 ? r : (r >> 1) & 7; };
    const int lr = lane / S::kRowChunks, lp = lane % S::kRowChunks;
    const char* xbase = rows + int64_t(row0) * pitch;
    auto load_x = [&](int32_t t, v4i* buf) {
#pragma unroll
        for (int j = 0; j < S::kRowLoads; ++j) {
            const int r = lr + j * S::kRowsPerLoad;
            if (j * S::kRowsPerLoad < nrows)
                load_to_lds(xbase + int64_t(t) * (S::kElems * 2),
                            static_cast<uint32_t>(min(r, nrows - 1) * pitch) + (lp ^ swz(r)) * 16,
                            buf + j * 64);
        }
    };
    f32x4 acc[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto compute = [&](const Weights<MXFP4> (&d)[kBlocks], const v4i* buf) {
#pragma unroll
        for (int s = 0; s < S::kProducts; ++s) {
            const bf16x8 fx =
                __builtin_bit_cast(bf16x8, buf[i * S::kRowChunks + ((4 * s + g) ^ swz(i))]);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
                acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(d[b].frag(s), fx, acc[b], 0, 0, 0);
        }
    };
    // Wavefront w takes steps w, w + kWaves, ...: the workgroup reads consecutive
    // weights. Two steps are in flight; LDS is this wavefront's own, so the
    // loop has no barrier.
    Weights<MXFP4> d0[kBlocks], d1[kBlocks];
    v4i* b0 = x0[wave];
    v4i* b1 = x1[wave];
    const int32_t n = full > wave ? (full - wave + kWaves - 1) / kWaves : 0;
    auto at = [&](int32_t k) { return wave + k * kWaves; };
    // A step's row loads go out before its weight loads, of which there are
    // kWeightLoads, and at least one row load: with the next step's behind
    // them, this step's rows have landed once no more than these are left.
    constexpr int kWeightLoads = 2 * kBlocks;
    auto load = [&](int32_t t, Weights<MXFP4> (&d)[kBlocks], v4i* buf) {
        wait_lds();           // the buffer's last reads have returned
        load_x(t, buf);
        __builtin_amdgcn_sched_barrier(0);
        load_w(t, d);
        __builtin_amdgcn_sched_barrier(0);
    };
    if (n > 0) {
        load(at(0), d0, b0);
        if (n > 1) load(at(1), d1, b1);
        int32_t k = 0;
        for (; k + 3 < n; k += 2) {
            wait_loads<kWeightLoads + 1>();
            compute(d0, b0);
            load(at(k + 2), d0, b0);
            wait_loads<kWeightLoads + 1>();
            compute(d1, b1);
            load(at(k + 3), d1, b1);
        }
        // One to three steps are left, the first two of them loaded.
        wait_loads<0>();
        compute(d0, b0);
        if (k + 2 < n) load(at(k + 2), d0, b0);
        if (k + 1 < n) compute(d1, b1);
        if (k + 2 < n) {
            wait_loads<0>();
            compute(d0, b0);
        }
    }
    // The last, partial step: row chunks past the row are zero, and so are the
    // weights there (packed weights hold zeros already).
    if (full < steps && wave == full % kWaves) {
        const v4i zero = {0, 0, 0, 0};
        const int32_t left = (red - full * S::kElems) / 8;
        wait_loads<0>();            // nothing still writes or reads b0
#pragma unroll
        for (int j = 0; j < S::kRowLoads; ++j) {
            const int r = lr + j * S::kRowsPerLoad;
            const int c = lp ^ swz(r);
            v4i v = zero;
            if (c < left)
                v = *reinterpret_cast<const v4i*>(xbase + min(r, nrows - 1) * pitch +
                                                  int64_t(full) * (S::kElems * 2) + c * 16);
            b0[j * 64 + lane] = v;
        }
        if constexpr (MXFP4) {
            load_w(full, d0);
        } else {
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    d0[b].q[s] = 4 * s + g < left ? *reinterpret_cast<const v4i*>(
                                                        wb[b] + int64_t(full) * 128 + s * 64)
                                                  : zero;
        }
        compute(d0, b0);
    }

    // Join the wavefronts' sums, in wavefront order.
    f32x4(*part)[kBlocks][64] =
        reinterpret_cast<f32x4(*)[kBlocks][64]>(MXFP4 ? &x0[0][0] : &sums[0][0]);
    wait_loads<0>();
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) part[wave][b][lane] = acc[b];
    __syncthreads();
    if (wave >= kFeatBlocks) return;
    f32x4 v = part[0][wave][lane];
    f32x4 u = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 1; p < kWaves; ++p) v += part[p][wave][lane];
    if constexpr (GATED) {
        u = part[0][wave + kFeatBlocks][lane];
#pragma unroll
        for (int p = 1; p < kWaves; ++p) u += part[p][wave + kFeatBlocks][lane];
    }
    const int32_t f = f0 + wave * 16 + g * 4;
    if (i >= nrows || f >= feats) return;
    v2i* o = reinterpret_cast<v2i*>(out + (int64_t(row0 + i) * feats + f) * 2);
    if constexpr (GATED) {
        f32x4 h;
#pragma unroll
        for (int t = 0; t < 4; ++t) h[t] = activate(act, v[t]) * u[t];
        *o = pack_bf16x4(h);
        if (pre) {
            float* p = pre + int64_t(row0 + i) * feats * 2 + f;
            *reinterpret_cast<f32x4*>(p) = v;
            *reinterpret_cast<f32x4*>(p + feats) = u;
        }
    } else {
        *o = pack_bf16x4(v);
    }
}

// One (feature, step) per thread: 64 bytes of values, rearranged from groups of
// 32 inputs into the lanes' 16 bytes, and the step's four scales. Lanes run
// over the 16 features of a block first, then over the steps, so that a
// wavefront reads 256 contiguous bytes of each feature and writes whole pieces
// of 256 bytes. Bound by those bytes: 256 experts of 7168 -> 4096 (8.0 GB) take
// 1.98 ms on MI355X, 4.0 TB/s.
__global__ __launch_bounds__(256)
void pack_mxfp4_kernel(const char* __restrict__ blocks, const uint8_t* __restrict__ scales,
                       int32_t N, int32_t K, int32_t nb, int32_t steps, int64_t tiles,
                       char* __restrict__ dst) {
    const int64_t q = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (q >= tiles * 16) return;
    const int i = static_cast<int>(q & 15);
    const int64_t tile = q >> 4;
    const int32_t t = static_cast<int32_t>(tile % steps);
    const int64_t eb = tile / steps;
    const int32_t f = 16 * static_cast<int32_t>(eb % nb) + i;
    const int64_t row = (eb / nb) * N + f;
    v4i v[4];
    uint32_t scale = 0x7F7F7F7Fu;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int32_t group = 4 * t + s;
        v[s] = v4i{0, 0, 0, 0};
        if (f < N && group < K / 32) {
            v[s] = *reinterpret_cast<const v4i*>(blocks + row * (K / 2) + group * 16);
            scale = (scale & ~(0xFFu << (8 * s))) |
                    (uint32_t(scales[row * (K / 32) + group]) << (8 * s));
        }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g)
        *reinterpret_cast<v4i*>(dst + tile * 1024 + (g * 16 + i) * 16) =
            v4i{v[0][g], v[1][g], v[2][g], v[3][g]};
    *reinterpret_cast<uint32_t*>(dst + tiles * 1024 + tile * 64 + i * 4) = scale;
}

int64_t stream_feature_tiles(const ExpertStreamArgs& a) {
    const int32_t per = (a.gated ? kBlocks / 2 : kBlocks) * 16;
    return (int64_t(a.feats) + per - 1) / per;
}

int64_t stream_workgroups(const ExpertStreamArgs& a) {
    const int64_t experts = a.max_rows < a.E ? a.max_rows : a.E;
    const int64_t tiles =
        stream_feature_tiles(a) * ((a.max_rows + kRows - 1) / kRows + experts);
    const int64_t unit = int64_t(kExpertXcds) * kXcdChunk;
    return (tiles + unit - 1) / unit * unit;
}

template <bool MXFP4, bool GATED>
hipError_t launch_stream(const ExpertStreamArgs& a, hipStream_t stream) {
    const char* w = static_cast<const char*>(a.w);
    const char* scales = w + mxfp4_tiles(a.E, a.gated ? 2 * a.feats : a.feats, a.red) * 1024;
    hipLaunchKernelGGL((expert_stream_kernel<MXFP4, GATED>),
                       dim3(static_cast<uint32_t>(stream_workgroups(a))),
                       dim3(waves_of(MXFP4) * 64), 0, stream, static_cast<const char*>(a.rows), w,
                       scales, a.offsets, a.E, static_cast<int32_t>(a.max_rows), a.red, a.feats,
                       static_cast<int32_t>(stream_feature_tiles(a)), a.activation,
                       static_cast<char*>(a.out), a.pre, a.zero);
    return hipGetLastError();
}

}  // namespace

int64_t expert_stream_grid(const ExpertStreamArgs& a) {
    return stream_workgroups(a) * (waves_of(a.mxfp4) * 64);
}

hipError_t launch_expert_stream(const ExpertStreamArgs& a, hipStream_t stream) {
    if (a.mxfp4)
        return a.gated ? launch_stream<true, true>(a, stream)
                       : launch_stream<true, false>(a, stream);
    return a.gated ? launch_stream<false, true>(a, stream) : launch_stream<false, false>(a, stream);
}

hipError_t launch_pack_mxfp4(const PackMxfp4Args& a, hipStream_t stream) {
    const int64_t tiles = mxfp4_tiles(a.E, a.N, a.K);
    hipLaunchKernelGGL(pack_mxfp4_kernel,
                       dim3(static_cast<uint32_t>(mxfp4_pack_grid(a.E, a.N, a.K) / 256)),
                       dim3(256), 0, stream, static_cast<const char*>(a.blocks),
                       static_cast<const uint8_t*>(a.scales), a.N, a.K, (a.N + 15) / 16,
                       (a.K + kMxfp4Step - 1) / kMxfp4Step, tiles, static_cast<char*>(a.dst));
    return hipGetLastError();
}

}  // namespace moe
