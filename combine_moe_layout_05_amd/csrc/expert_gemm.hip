// Products of the gated expert feed-forward block on gfx950, and their
// gradients with respect to the rows: grouped GEMMs over the expert-major rows
// with the block's element-wise part in the epilogue. With rows r of expert e,
//     kGated      g = x[r] Wg^T, u = x[r] Wu^T, out[r] = act(g) * u
//     kPlain      out[r] = x[r] W^T
//     kInputGrad  out[r] = dy[r] W
//     kGatedGrad  dh = dy[r] Wd, out[r] = [dh * u * act'(g) | dh * act(g)]
// The matrix cores take 16 weight positions x 16 rows x 32 of the sum at a
// time, weights as the first operand, so a lane ends up with four neighbouring
// features of one row and writes them together.
//
// Bound. A segment's weights are read once per row tile, so up to a few hundred
// rows per expert the weights' bytes count, above that the matrix cores. A
// 256 x 256 tile takes (256 + 256) * 2 bytes from the L2 cache per 256 * 256 * 2
// operations, 128 operations a byte: 11 TB/s at 1.44 PFLOP/s, which the caches
// hold only because the tiles of an XCD share operands (chunks of 16 tile
// numbers in bands of 8 row tiles; with chunks of 32 or 64 the L2 caches read
// 4 to 6 % less, which gains nothing at 512 rows per expert and loses up to 15 %
// at 128, where the last chunks leave XCDs idle).
// Eight wavefronts of 64 x 128 make it, one workgroup to a CU: their sums take
// half the registers, the fragments of two half steps most of the rest.
//
// Measured on MI355X (a large library product reaches 1438 TFLOP/s, a large
// copy 4.9 TB/s), two cards. 128 experts, 4096 -> 2 x 2048, 65536 rows routed at
// random (512 per expert on average; some 60 experts end in a tile of at most 64
// rows, 318 row tiles where the rows fill 256) and, behind the bar, exactly 512
// rows per expert: gated 2.27 to 2.35 | 2.06 to 2.12 ms with the fp32 projections
// written out for the backward (0.94 to 0.97 PFLOP/s and 1 GB of them), 2.10 to
// 2.19 | 1.87 to 1.94 without, the second projection 1.11 to 1.15 | 1.00 to 1.04
// (0.96 to 0.99 PFLOP/s), its gate gradient 1.33 to 1.39 | 1.19 to 1.21 (0.79 to
// 0.83), the input gradient 2.08 to 2.24 | 1.89 to 1.97 (0.98 to 1.06). One expert of
// 65536 rows: 1.27 to 1.34 PFLOP/s. 256 experts of 128 rows on average, skewed,
// 7168 -> 2 x 2048: 3.28 to 3.37 ms for 15.6 GB (4.7 TB/s); of 2 rows: 1.36 to 1.38
// ms for 8.0 GB (5.8 TB/s). LDS bank conflicts count 0; in the routed case the
// matrix cores are busy 58 % of the cycles at a clock that power holds near 1.7
// GHz, while 10 GB pass behind the L2 caches in 2.1 ms.
#include "expert_kernels.h"
#include "expert_mma.h"

namespace moe {
namespace {

constexpr int kWavesR = 2;              // wavefronts along the rows
constexpr int kBlkF = 4;                // 16-position blocks of weights per wavefront

// A workgroup's tile: WAVES_F pairs of wavefronts, 64 weight positions each,
// times ROWS rows. The large one reads least per product; the small one makes up
// to eight times as many workgroups of the same product, two to a CU.
template <int WAVES_F, int ROWS>
struct Shape {
    static constexpr int kWavesF = WAVES_F;
    static constexpr int kWaves = WAVES_F * kWavesR;
    static constexpr int kTileF = WAVES_F * kBlkF * 16;
    static constexpr int kTileR = ROWS;
    // Stages of 64-element steps in LDS for a tile of `rows` rows. A third stage
    // of the weights beside two of 256 rows (160 KiB) gave 0.8 % where the
    // weights' bytes count and cost 2 to 4 % where the matrix cores do.
    static constexpr int stages(int rows) { return rows > 128 ? 2 : 3; }
    // Output features: the gated product holds gate and up rows.
    static constexpr int feats(ExpertOp op) { return op == ExpertOp::kGated ? kTileF / 2 : kTileF; }
};
typedef Shape<4, 256> Large;
typedef Shape<2, 64> Small;
constexpr int kXcdChunk = 16;
constexpr int kBand = 8;

constexpr bool strided(ExpertOp op) {
    return op == ExpertOp::kInputGrad || op == ExpertOp::kGatedGrad;
}

template <class S, bool STRIDED>
struct WeightOperand {
    typedef PackedOperand<S::kTileF, S::kWaves> type;
};
template <class S>
struct WeightOperand<S, true> {
    typedef StridedOperand<S::kTileF, S::kWaves, 64> type;
};

template <ExpertOp OP, class S>
__global__ __launch_bounds__(S::kWaves * 64, 2)
void expert_gemm_kernel(const char* __restrict__ rows, const char* __restrict__ w,
                        const int32_t* __restrict__ offsets, int32_t E, int32_t max_rows,
                        int32_t red, int32_t feats, int32_t ftiles, int32_t act,
                        char* __restrict__ out, float* __restrict__ pre, int32_t zero) {
    constexpr int kWaves = S::kWaves, kWavesF = S::kWavesF, kTileF = S::kTileF,
                  kTileR = S::kTileR;
    typedef typename WeightOperand<S, strided(OP)>::type Weights;
    constexpr auto lds_of = [](int rows) {
        return S::stages(rows) * (Weights::kChunks + rows * 8);
    };
    constexpr int kHalf = kTileR > 64 ? kTileR / 2 : kTileR;
    __shared__ v4i lds[lds_of(kHalf) > lds_of(kTileR) ? lds_of(kHalf) : lds_of(kTileR)];
    __shared__ int32_t info[4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    const int64_t number = expert_tile_number(kXcdChunk);
    if (wave == 0) {
        const ExpertTile t =
            expert_find_tile(offsets, E, max_rows, kTileR, ftiles, kBand, number);
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
    const int64_t out_pitch = int64_t(feats) * (OP == ExpertOp::kGatedGrad ? 4 : 2);
    if (e < 0) {
        if (zero)
            expert_zero_rows(reinterpret_cast<v4i*>(out), offsets, zero, row0, max_rows,
                             static_cast<int32_t>(out_pitch / 16), ft, int64_t(gridDim.x) - nrows);
        return;
    }
    const int32_t f0 = ft * S::feats(OP);
    const int64_t red_pitch = int64_t(red) * 2;

    const int wf = wave % kWavesF, wr = wave / kWavesF;
    Weights wt;
    if constexpr (strided(OP)) {
        // w[e] is [red][feats], features contiguous.
        const char* base = w + (int64_t(e) * red * feats + f0) * 2;
        wt.init(wave, lane, wf * kBlkF, int64_t(feats) * 2, base, min(kTileF, feats - f0));
    } else if constexpr (OP == ExpertOp::kGated) {
        // Each wavefront's 64 positions are 32 gate rows and the 32 up rows of
        // the same features, so the epilogue finds both in its own registers.
        const char* gate = w + (int64_t(e) * 2 * feats + f0) * red_pitch;
        const char* up = gate + int64_t(feats) * red_pitch;
        const int last = feats - f0 - 1;
        wt.init(wave, lane, wf * kBlkF, red_pitch, [&](int p0) { return (p0 & 32) ? up : gate; },
                [&](int p) { return min((p >> 6) * 32 + (p & 31), last); });
    } else {
        const char* base = w + (int64_t(e) * feats + f0) * red_pitch;
        const int last = feats - f0 - 1;
        wt.init(wave, lane, wf * kBlkF, red_pitch, [&](int) { return base; },
                [&](int p) { return min(p, last); });
    }
    // Experts begin their sums at different steps. Rows of weights whose pitch is a
    // power of two have equal steps in few channels of the caches and of HBM, and
    // workgroups started together read equal steps: 128 experts of 128 rows, 2048 ->
    // 2 x 1408 gated, 366 us without this and 310 with it, 64 of 128 rows, 2048 ->
    // 7168, 456 and 378, 32 of 30 rows, 2048 -> 2 x 1024, 64 and 53; within 2 % at
    // other pitches. The gradients read a step as whole rows and lose 2 %; starting
    // every feature tile elsewhere loses what the tiles share in the L2 cache (1
    // to 6 %).
    const int32_t first = strided(OP) ? 0 : e * 5 % max(red / 64, 1);
    // The loop exists for each 64-row count up to the tile's and is chosen once
    // per workgroup, so that a segment's last tile costs what its rows need.
    auto run = [&](auto parts) {
        constexpr int kRowsUsed = decltype(parts)::value * 64;
        constexpr int kBlkR = kRowsUsed / kWavesR / 16;
        constexpr int kStages = S::stages(kRowsUsed);
        PackedOperand<kRowsUsed, kWaves> rt;
        const char* rbase = rows + int64_t(row0) * red_pitch;
        rt.init(wave, lane, wr * kBlkR, red_pitch, [&](int) { return rbase; },
                [&](int p) { return min(p, nrows - 1); });
        f32x4 acc[kBlkF][kBlkR];
        typedef Accumulator<kStages, kBlkF, kBlkR, Weights, PackedOperand<kRowsUsed, kWaves>> Sums;
        const Sums sums{lds, lane, first, red / 64};
        sums.run(wt, rt, red, acc);

        // acc[a][b][t] belongs to row 16b + lane % 16 and position 16a + 4 (lane /
        // 16) + t of the wavefront.
        const int i = lane & 15, g = lane >> 4;
    #pragma unroll
        for (int b = 0; b < kBlkR; ++b) {
            const int r = (wr * kBlkR + b) * 16 + i;
            if (r >= nrows) continue;
            char* orow = out + int64_t(row0 + r) * out_pitch;
            // Two 16-feature blocks at a time: every lane ends up with eight
            // neighbouring features, which begin `at` features into the pair.
            const int at = (g & 1) * 16 + (g >> 1) * 8;
            // Each result is rounded to bf16 here, once: h and the gradient of [g | u]
            // are operands of the matrix-core products that follow, which take
            // bf16; with more bits each would be two operands, at twice the products.
            // [g | u], which only the epilogue of the gate gradient reads, is kept in
            // fp32.
            if constexpr (OP == ExpertOp::kGated) {
                static_assert(kBlkF == 4, "a pair of gate blocks, then their up blocks");
                const int32_t f = f0 + wf * 32;
                v2i h[2];
    #pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const f32x4 gv = acc[a][b], uv = acc[a + 2][b];
                    f32x4 v;
    #pragma unroll
                    for (int t = 0; t < 4; ++t) v[t] = activate(act, gv[t]) * uv[t];
                    h[a] = pack_bf16x4(v);
                    const int32_t fq = f + a * 16 + g * 4;
                    if (pre && fq < feats) {
                        float* p = pre + int64_t(row0 + r) * feats * 2 + fq;
                        *reinterpret_cast<f32x4*>(p) = gv;
                        *reinterpret_cast<f32x4*>(p + feats) = uv;
                    }
                }
                const v4i v = pair_blocks(h[0], h[1]);
                if (f + at < feats) *reinterpret_cast<v4i*>(orow + int64_t(f + at) * 2) = v;
            } else {
    #pragma unroll
                for (int a = 0; a < kBlkF; a += 2) {
                    const int32_t f = f0 + (wf * kBlkF + a) * 16;
                    if constexpr (OP == ExpertOp::kGatedGrad) {
                        v2i dg[2], du[2];
    #pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int32_t fq = min(f + c * 16 + g * 4, feats - 4);
                            const float* p = pre + int64_t(row0 + r) * feats * 2 + fq;
                            const f32x4 gv = *reinterpret_cast<const f32x4*>(p);
                            const f32x4 uv = *reinterpret_cast<const f32x4*>(p + feats);
                            const f32x4 v = acc[a + c][b];
                            f32x4 vg, vu;
    #pragma unroll
                            for (int t = 0; t < 4; ++t) {
                                float value, slope;
                                activate_grad(act, gv[t], value, slope);
                                vg[t] = v[t] * uv[t] * slope;
                                vu[t] = v[t] * value;
                            }
                            dg[c] = pack_bf16x4(vg);
                            du[c] = pack_bf16x4(vu);
                        }
                        const v4i og = pair_blocks(dg[0], dg[1]), ou = pair_blocks(du[0], du[1]);
                        if (f + at < feats) {
                            *reinterpret_cast<v4i*>(orow + int64_t(f + at) * 2) = og;
                            *reinterpret_cast<v4i*>(orow + (int64_t(feats) + f + at) * 2) = ou;
                        }
                    } else {
                        const v4i v =
                            pair_blocks(pack_bf16x4(acc[a][b]), pack_bf16x4(acc[a + 1][b]));
                        if (f + at < feats) *reinterpret_cast<v4i*>(orow + int64_t(f + at) * 2) = v;
                    }
                }
            }
        }
    };
    const int parts = (nrows + 63) / 64;
    if constexpr (kTileR > 64) {
        if (parts == 2) return run(std::integral_constant<int, 2>{});
        if (parts == 3) return run(std::integral_constant<int, 3>{});
        if (parts == 4) return run(std::integral_constant<int, 4>{});
    }
    run(std::integral_constant<int, 1>{});
}

template <class S>
int64_t feature_tiles(ExpertOp op, int32_t feats) {
    const int32_t per = S::feats(op);
    return (int64_t(feats) + per - 1) / per;
}

template <class S>
int64_t grid_of(const ExpertGemmArgs& a) {
    // A segment of c rows takes ceil(c / kTileR) row tiles, at most one more
    // per expert with rows than the rows fill.
    const int64_t experts = a.max_rows < a.E ? a.max_rows : a.E;
    const int64_t tiles =
        feature_tiles<S>(a.op, a.feats) * ((a.max_rows + S::kTileR - 1) / S::kTileR + experts);
    const int64_t unit = int64_t(kExpertXcds) * kXcdChunk;
    return (tiles + unit - 1) / unit * unit;
}

}  // namespace

// The small shape where segments are short, or where the large one would leave
// half the 256 CUs idle. Measured on MI355X, weights from HBM, large against
// small:
//   - 8 rows per expert, skewed, 256 experts of 7168 -> 2 x 2048 gated 2371 and
//     2248 us; 32 rows, skewed, 128 experts of 2048 -> 2 x 1408 353 and 292, its
//     gradients towards the rows 213 and 158, 287 and 278; 256 experts 2597 and
//     2610. At 64 rows 383 and 341 but 2771 and 2980.
//   - one expert of 4096 -> 2 x 2048 gated: 98.6 and 34.2 us at 512 rows (32
//     large tiles), 100 and 104 at 2048 (128), 135 and 201 at 4096 (256); 8 of
//     100 rows 80.4 and 71.8 (128); 24 of 1992 -> 2 x 1000 60.7 and 70.1 at 92
//     rows (192).
bool expert_small_tile(ExpertOp op, int32_t E, int64_t max_rows, int32_t feats) {
    if (max_rows <= int64_t(32) * E) return true;
    const int64_t row_tiles = (max_rows + Large::kTileR - 1) / Large::kTileR;
    const int64_t experts = max_rows < E ? max_rows : E;
    return feature_tiles<Large>(op, feats) * (row_tiles > experts ? row_tiles : experts) <= 128;
}

namespace {

bool small_tile(const ExpertGemmArgs& a) {
    return expert_small_tile(a.op, a.E, a.max_rows, a.feats);
}

template <ExpertOp OP, class S>
hipError_t launch_shape(const ExpertGemmArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((expert_gemm_kernel<OP, S>), dim3(static_cast<uint32_t>(grid_of<S>(a))),
                       dim3(S::kWaves * 64), 0, stream, static_cast<const char*>(a.rows),
                       static_cast<const char*>(a.w), a.offsets, a.E,
                       static_cast<int32_t>(a.max_rows), a.red, a.feats,
                       static_cast<int32_t>(feature_tiles<S>(a.op, a.feats)), a.activation,
                       static_cast<char*>(a.out), a.pre, a.zero);
    return hipGetLastError();
}

template <ExpertOp OP>
hipError_t launch_op(const ExpertGemmArgs& a, hipStream_t stream) {
    return small_tile(a) ? launch_shape<OP, Small>(a, stream) : launch_shape<OP, Large>(a, stream);
}

}  // namespace

int64_t expert_gemm_grid(const ExpertGemmArgs& a) {
    return small_tile(a) ? grid_of<Small>(a) * (Small::kWaves * 64)
                        : grid_of<Large>(a) * (Large::kWaves * 64);
}

hipError_t launch_expert_gemm(const ExpertGemmArgs& a, hipStream_t stream) {
    switch (a.op) {
        case ExpertOp::kPlain: return launch_op<ExpertOp::kPlain>(a, stream);
        case ExpertOp::kGated: return launch_op<ExpertOp::kGated>(a, stream);
        case ExpertOp::kInputGrad: return launch_op<ExpertOp::kInputGrad>(a, stream);
        default: return launch_op<ExpertOp::kGatedGrad>(a, stream);
    }
}

}  // namespace moe
