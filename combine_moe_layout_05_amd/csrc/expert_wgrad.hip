// Gradient of the expert weights on gfx950: for every expert e
//     dw[e][n][k] = sum over rows r of e's segment of dy[r][n] * x[r][k]
// (plus what dw holds, on request), one rounding of the fp32 sum.
#include "expert_kernels.h"
#include "expert_mma.h"

namespace moe {
namespace {

constexpr int kWaves = 8;
constexpr int kWavesK = 4;
constexpr int kWavesN = 2;
constexpr int kTileK = 256;
constexpr int kTileN = 256;
constexpr int kBlkK = kTileK / kWavesK / 16;
constexpr int kBlkN = kTileN / kWavesN / 16;
constexpr int kXcdChunk = 32;

template <bool F32, bool ACCUMULATE>
__global__ __launch_bounds__(kWaves * 64, 2)
void expert_wgrad_kernel(const char* __restrict__ dy, const char* __restrict__ x,
                         const int32_t* __restrict__ offsets, int32_t max_rows, int32_t N,
                         int32_t K, int32_t ntiles, int32_t ktiles, int32_t strip, int64_t tiles, char* __restrict__ dw) {
    typedef StridedOperand<kTileK, kWaves> Kop;
    typedef StridedOperand<kTileN, kWaves> Nop;
    typedef Accumulator<2, kBlkK, kBlkN, Kop, Nop> Sums;
    __shared__ v4i lds[Sums::kLdsChunks];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t u = expert_tile_number(kXcdChunk);
    if (u >= tiles) return;
    const int32_t strips = (ktiles + strip - 1) / strip;
    const int32_t per = ntiles * strips;
    const int32_t e = static_cast<int32_t>(u / per);
    const int32_t in = static_cast<int32_t>(u - int64_t(e) * per);
    const int32_t nt0 = (in / strips) * kTileN;
    const int32_t first = (in % strips) * strip;
    const int32_t end = min(first + strip, ktiles);
    int32_t s0, s1;
    expert_segment(offsets, e, max_rows, s0, s1);
    const int32_t count = s1 - s0;
    if (ACCUMULATE && count == 0) return;

    Kop ko;
    Nop no;
    const int wk = wave % kWavesK, wn = wave / kWavesK;
    auto at_tile = [&](int32_t t) {
        ko.init(wave, lane, wk * kBlkK, int64_t(K) * 2,
                x + (int64_t(s0) * K + int64_t(t) * kTileK) * 2, min(kTileK, K - t * kTileK));
    };
    no.init(wave, lane, wn * kBlkN, int64_t(N) * 2, dy + (int64_t(s0) * N + nt0) * 2,
            min(kTileN, N - nt0));
    f32x4 acc[kBlkK][kBlkN];
    const Sums sums{lds, lane};
    at_tile(first);
    sums.start(ko, no, count);
    constexpr int kStores = kBlkK * kBlkN / (F32 ? 1 : 2);
    bool whole = false;     // the previous tile's stores went out in full
    for (int32_t t = first; t < end; ++t) {
    const int32_t kt0 = t * kTileK;
    // The next tile's first loads are in flight while this one is stored, and
    // its first products run while the stores drain.
    sums.template run<(ACCUMULATE ? 0 : kStores)>(ko, no, count, whole, acc);
    if (t + 1 < end) {
        at_tile(t + 1);
        sums.start(ko, no, count);
    }
    whole = nt0 + kTileN <= N && kt0 + kTileK <= K;

    const int i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int b = 0; b < kBlkN; ++b) {
        const int32_t n = nt0 + (wn * kBlkN + b) * 16 + i;
        if (n >= N) continue;
        const int64_t row = (int64_t(e) * N + n) * K;
#pragma unroll
        for (int a = 0; a < kBlkK; a += 2) {
            if constexpr (F32) {
#pragma unroll
                for (int c = a; c < a + 2; ++c) {
                    const int32_t k = kt0 + (wk * kBlkK + c) * 16 + g * 4;
                    if (k >= K) continue;
                    f32x4* p = reinterpret_cast<f32x4*>(dw + (row + k) * 4);
                    f32x4 v = acc[c][b];
                    if constexpr (ACCUMULATE) v = *p + v;
                    *p = v;
                }
            } else if constexpr (ACCUMULATE) {
#pragma unroll
                for (int c = a; c < a + 2; ++c) {
                    const int32_t k = kt0 + (wk * kBlkK + c) * 16 + g * 4;
                    if (k >= K) continue;
                    v2i* p = reinterpret_cast<v2i*>(dw + (row + k) * 2);
                    f32x4 v = acc[c][b];
                    const v2i o = *p;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t word = static_cast<uint32_t>(o[q >> 1]);
                        v[q] += (q & 1) ? bf16_hi(word) : bf16_lo(word);
                    }
                    *p = pack_bf16x4(v);
                }
            } else {
                const int32_t k = kt0 + (wk * kBlkK + a + (g & 1)) * 16 + (g >> 1) * 8;
                const v4i v = pair_blocks(pack_bf16x4(acc[a][b]), pack_bf16x4(acc[a + 1][b]));
                if (k < K) *reinterpret_cast<v4i*>(dw + (row + k) * 2) = v;
            }
        }
    }
    }
}

int32_t k_tiles(const ExpertWgradArgs& a) {
    return static_cast<int32_t>((int64_t(a.K) + kTileK - 1) / kTileK);
}
int32_t n_tiles(const ExpertWgradArgs& a) {
    return static_cast<int32_t>((int64_t(a.N) + kTileN - 1) / kTileN);
}
// Tiles along K per workgroup.
int32_t strip_of(const ExpertWgradArgs& a) {
    const int64_t tiles = int64_t(n_tiles(a)) * k_tiles(a) * a.E;
    return tiles >= 8192 ? 4 : tiles >= 2048 ? 2 : 1;
}
int64_t strip_count(const ExpertWgradArgs& a) {
    const int32_t strip = strip_of(a);
    return int64_t(n_tiles(a)) * ((k_tiles(a) + strip - 1) / strip) * a.E;
}

}  // namespace

int64_t expert_wgrad_grid(const ExpertWgradArgs& a) {
    const int64_t unit = int64_t(kExpertXcds) * kXcdChunk;
    return (strip_count(a) + unit - 1) / unit * unit;
}

hipError_t launch_expert_wgrad(const ExpertWgradArgs& a, hipStream_t stream) {
    auto kernel = a.f32 ? (a.accumulate ? expert_wgrad_kernel<true, true> : expert_wgrad_kernel<true, false>)
                        : (a.accumulate ? expert_wgrad_kernel<false, true> : expert_wgrad_kernel<false, false>);
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(expert_wgrad_grid(a))),
                       dim3(kWaves * 64), 0, stream, static_cast<const char*>(a.dy),
                       static_cast<const char*>(a.x), a.offsets, static_cast<int32_t>(a.max_rows),
                       a.N, a.K, n_tiles(a), k_tiles(a), strip_of(a), strip_count(a),
                       static_cast<char*>(a.dw));
    return hipGetLastError();
}

}  // namespace moe
