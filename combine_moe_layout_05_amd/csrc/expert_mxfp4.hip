// Expert products with packed 4-bit weights for many rows per expert on
// gfx950: out[r] = x[r] W^T, or act(g) * u of the two projections.
//
// The rows are bf16, so the weights become bf16 too (exactly: 2-bit significands
// times a power of two) in the registers of the wavefront that multiplies them,
// four conversions to 8 weights. A wavefront keeps its 64 features' weights to
// itself, 4 KiB a step, read from HBM or L2 straight into the registers two
// steps ahead; the rows, which all wavefronts share, go through LDS. At 64 rows
// there is one conversion to a product, vector work that runs beside it.
//
// Bound: the weights' bytes below some 100 rows per expert, then the matrix
// cores. Measured on MI355X at 256 experts of 128 rows on average, skewed, 7168
// -> 2 x 2048: 1.80 to 1.88 ms, 1.02 to 1.07 PFLOP/s, the matrix cores busy 66 % of
// the cycles, LDS bank conflicts 0; 2048 -> 7168 0.98 ms. Chunks of 16 to 128 tile
// numbers instead of 8 read up to 15 % less behind the L2 caches (11.7 GB at 8) in
// the same time (1 %).
#include "expert_kernels.h"
#include "expert_mma.h"
#include "expert_mxfp4.h"

namespace moe {
namespace {

constexpr int kBlocks = 4;              // 16-feature blocks per wavefront

// Four wavefronts and 64 rows: two such workgroups fit a CU. Measured on MI355X
// against eight wavefronts of 128 rows, one to a CU, and two of 64 rows: 43.8
// against 90.9 and 52.4 us for one expert of 4096 -> 2 x 2048 at 1024 rows, 569
// against 597 and 695 us for 128 such experts at 16384 rows, 971 against 976 and
// 1214 us at 32768.
constexpr int kWaves = 4;               // along the features
constexpr int kRowTile = 64;
constexpr int kStages = 3;              // 128-element steps of rows in LDS
constexpr int kXcdChunk = 8;
constexpr int kBand = 8;

template <bool GATED>
__global__ __launch_bounds__(kWaves * 64, 2)
void expert_mxfp4_kernel(const char* __restrict__ rows, const char* __restrict__ w,
                         const char* __restrict__ scales, const int32_t* __restrict__ offsets,
                         int32_t E, int32_t max_rows, int32_t red, int32_t feats, int32_t ftiles,
                         int32_t act, char* __restrict__ out, int32_t zero) {
    // Output features of a wavefront: half its blocks are up rows if gated.
    constexpr int kFeats = kBlocks * 16 / (GATED ? 2 : 1);
    __shared__ v4i lds[kStages * 2 * PackedOperand<kRowTile, kWaves>::kChunks];
    __shared__ int32_t info[4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t number = expert_tile_number(kXcdChunk);
    if (wave == 0) {
        const ExpertTile t =
            expert_find_tile(offsets, E, max_rows, kRowTile, ftiles, kBand, number);
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
    const int32_t f0 = (ft * kWaves + wave) * kFeats;
    const int32_t steps = (red + kMxfp4Step - 1) / kMxfp4Step;

    // This wavefront's blocks; those past the matrix read its last one and are
    // not stored.
    const char* wb[kBlocks];
    const char* sb[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        const int32_t nb = (feats + 15) / 16;
        const bool up = GATED && b >= kBlocks / 2;
        const int32_t ob = min(f0 / 16 + (GATED ? b % (kBlocks / 2) : b), nb - 1);
        const int64_t blk = (int64_t(e) * (GATED ? 2 : 1) + (up ? 1 : 0)) * nb + ob;
        wb[b] = w + blk * steps * 1024;
        sb[b] = scales + blk * steps * 64;
    }

    auto run = [&](auto row_blocks) {
        constexpr int NB = decltype(row_blocks)::value;
        typedef PackedOperand<kRowTile, kWaves> Rows;
        constexpr int kLoads = 2 * Rows::kLoads;                // of a step
        Rows rt;
        const int64_t pitch = int64_t(red) * 2;
        const char* rbase = rows + int64_t(row0) * pitch;
        rt.init(wave, lane, 0, pitch, [&](int) { return rbase; },
                [&](int p) { return min(p, nrows - 1); });
        f32x4 acc[kBlocks][NB];
#pragma unroll
        for (int a = 0; a < kBlocks; ++a)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        auto stage_of = [&](int stage) { return lds + stage * 2 * Rows::kChunks; };
        // Rows of step t: two operand steps of 64, the last possibly partial
        // (the halves past the row read its beginning and become zero).
        auto issue_rows = [&](int32_t t, int stage) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int left = min(red - (2 * t + h) * 64, 64);
                v4i* buf = stage_of(stage) + h * Rows::kChunks;
                if (left == 64)
                    rt.issue(2 * t + h, buf);
                else
                    rt.issue_partial(left > 0 ? 2 * t + h : 0, max(left, 0), lane, buf);
            }
        };
        auto load_w = [&](int32_t t, Mxfp4Step (&d)[kBlocks]) {
            // A uniform address and a 32-bit offset per lane (a register, not
            // an address pair per load).
            uint32_t qo = lane * 16, so = i * 4;
            reform(qo);
            reform(so);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                d[b].q = *reinterpret_cast<const v4i*>(wb[b] + int64_t(t) * 1024 + qo);
                d[b].scale = *reinterpret_cast<const uint32_t*>(sb[b] + int64_t(t) * 64 + so);
            }
        };
        // Zeros into what the loads of step t put past the rows' end, or into
        // all of a step that does not exist (an odd number of them ends with
        // one of zeros).
        auto clear = [&](int32_t t, int stage) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int left = min(red - (2 * t + h) * 64, 64);
                if (left < 64) rt.fix(max(left, 0), lane, stage_of(stage) + h * Rows::kChunks);
            }
            wait_lds();
            step_barrier();
        };
        const bool partial = red % kMxfp4Step != 0;

        Mxfp4Step even[kBlocks], odd[kBlocks];
        issue_rows(0, 0);
        if (steps > 1) issue_rows(1, 1);
        load_w(0, even);
        load_w(min(1, steps - 1), odd);
        wait_loads<4 * kBlocks>();
        step_barrier();
        if (partial && steps == 1) clear(0, 0);
        int stage = 0;
        auto step = [&](Mxfp4Step (&mine)[kBlocks], int32_t t) {
            const int after = stage + 1 == kStages ? 0 : stage + 1;
            const int free = after + 1 == kStages ? 0 : after + 1;
            bf16x8 wf[kBlocks];
#pragma unroll
            for (int a = 0; a < kBlocks; ++a) wf[a] = mine[a].frag(0);
            __builtin_amdgcn_sched_barrier(0);
            // Behind the first use of this step's weights: what waits for them
            // must not wait for these loads.
            if (t + 2 < steps) issue_rows(t + 2, free);
            const v4i* buf = stage_of(stage);
            // The rows of scale group s, one product deep.
            auto fetch = [&](int s, bf16x8 (&d)[NB]) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    d[b] = rt.frag(buf + (s >> 1) * Rows::kChunks, b, s & 1);
            };
            bf16x8 cur[NB], nxt[NB];
            fetch(0, cur);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s < 3) fetch(s + 1, nxt);
                if (s > 0) {
#pragma unroll
                    for (int a = 0; a < kBlocks; ++a) wf[a] = mine[a].frag(s);
                }
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int a = 0; a < kBlocks; ++a)
                        acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[a], cur[b],
                                                                            acc[a][b], 0, 0, 0);
#pragma unroll
                for (int b = 0; b < NB; ++b) cur[b] = nxt[b];
            }
            __builtin_amdgcn_sched_barrier(0);
            load_w(min(t + 2, steps - 1), mine);
            __builtin_amdgcn_sched_barrier(0);
            // The next step's rows have landed: behind them are two steps'
            // weights and the rows of the step after it, if there are any.
            if (t + 2 < steps)
                wait_loads<kLoads + 4 * kBlocks>();
            else
                wait_loads<4 * kBlocks>();
            step_barrier();
            if ((partial && t + 2 == steps) || t + 1 == steps) clear(t + 1, after);
            stage = after;
        };
        for (int32_t t = 0; t < steps; t += 2) {
            step(even, t);
            if (t + 1 >= steps) {
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) odd[b].q = v4i{0, 0, 0, 0};
            }
            step(odd, t + 1);
        }
        wait_loads<0>();

        const int at = (g & 1) * 16 + (g >> 1) * 8;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int r = b * 16 + i;
            if (r >= nrows) continue;
            char* orow = out + int64_t(row0 + r) * feats * 2;
            if constexpr (GATED) {
                v2i h[2];
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    f32x4 v;
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        v[t] = activate(act, acc[a][b][t]) * acc[a + 2][b][t];
                    h[a] = pack_bf16x4(v);
                }
                const v4i v = pair_blocks(h[0], h[1]);
                if (f0 + at < feats) *reinterpret_cast<v4i*>(orow + int64_t(f0 + at) * 2) = v;
            } else {
#pragma unroll
                for (int a = 0; a < kBlocks; a += 2) {
                    const int32_t f = f0 + a * 16 + at;
                    const v4i v = pair_blocks(pack_bf16x4(acc[a][b]), pack_bf16x4(acc[a + 1][b]));
                    if (f < feats) *reinterpret_cast<v4i*>(orow + int64_t(f) * 2) = v;
                }
            }
        }
    };
    // Short last tiles cost what their rows need.
    if (nrows <= 16)
        run(std::integral_constant<int, 1>{});
    else if (nrows <= 32)
        run(std::integral_constant<int, 2>{});
    else if (nrows <= 48)
        run(std::integral_constant<int, 3>{});
    else
        run(std::integral_constant<int, 4>{});
}

int64_t feature_tiles(const ExpertStreamArgs& a) {
    const int32_t per = kWaves * kBlocks * 16 / (a.gated ? 2 : 1);
    return (int64_t(a.feats) + per - 1) / per;
}

int64_t grid_of(const ExpertStreamArgs& a) {
    const int64_t experts = a.max_rows < a.E ? a.max_rows : a.E;
    const int64_t tiles = feature_tiles(a) * ((a.max_rows + kRowTile - 1) / kRowTile + experts);
    const int64_t unit = int64_t(kExpertXcds) * kXcdChunk;
    return (tiles + unit - 1) / unit * unit;
}

}  // namespace

int64_t expert_mxfp4_grid(const ExpertStreamArgs& a) { return grid_of(a) * (kWaves * 64); }

hipError_t launch_expert_mxfp4(const ExpertStreamArgs& a, hipStream_t stream) {
    const char* w = static_cast<const char*>(a.w);
    const char* scales = w + mxfp4_tiles(a.E, a.gated ? 2 * a.feats : a.feats, a.red) * 1024;
    auto kernel = a.gated ? expert_mxfp4_kernel<true> : expert_mxfp4_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(grid_of(a))),
                       dim3(kWaves * 64), 0, stream, static_cast<const char*>(a.rows), w, scales,
                       a.offsets, a.E, static_cast<int32_t>(a.max_rows), a.red, a.feats,
                       static_cast<int32_t>(feature_tiles(a)), a.activation,
                       static_cast<char*>(a.out), a.zero);
    return hipGetLastError();
}

}  // namespace moe
