// Expert products of 4-bit rows with packed 4-bit weights on gfx950: out[r] =
// x[r] W^T, or act(g) * u of the two projections, both operands e2m1 with a
// power-of-two scale per 32 elements of the sum, which the matrix cores apply
// themselves.
//
// A matrix-core product takes 128 elements of the sum; lane (i, g) of an operand
// holds position i's 32 values of scale group g, and that group's scale. Rows lie
// in memory that way (16 bytes per group). The packed weights, which the products
// with bf16 rows share, hold 8 values of each of the four groups in a lane: a
// transpose of 4 x 4 dwords between the lanes of a feature (four register swaps)
// puts them in place.
//
// Elements past the end of a sum meet weights of zero, which the packing put
// there; what is read in their place is finite, or makes the row NaN anyway.
#include "expert_kernels.h"
#include "expert_mma.h"
#include "layer_kernels.h"

namespace moe {
namespace {

typedef int32_t v8i __attribute__((ext_vector_type(8)));

constexpr int kBlocks = 4;              // 16-feature blocks per wavefront

// c + a b over 128 elements; a's scale is the low byte of sa, b's byte BYTE of sb.
template <int BYTE>
__device__ __forceinline__ f32x4 multiply4(v4i a, int32_t sa, v4i b, int32_t sb, f32x4 c) {
    const v8i wa = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
    const v8i wb = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, wb, c, 4, 4, 0, sa, BYTE, sb);
}

// Packed weights to an operand: dword s of lane group g and dword g of lane
// group s change places.
__device__ __forceinline__ v4i by_groups(v4i q) {
    const auto a = __builtin_amdgcn_permlane32_swap(q[0], q[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(q[1], q[3], false, false);
    const auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return v4i{static_cast<int32_t>(lo[0]), static_cast<int32_t>(lo[1]),
               static_cast<int32_t>(hi[0]), static_cast<int32_t>(hi[1])};
}

// ---- Many rows per expert -------------------------------------------------
//
// A wavefront keeps 64 features' weights to itself, straight from memory into
// registers; the rows, which the workgroup's four wavefronts share, go through LDS,
// and so do their scales, all of a tile's at its start.
//
// What bounds it where rows are many: the waits of a step. The branch between a
// step's two halves ends a block of code, and the compiler moves the first half's
// products past it: as built, all 64 products of a wavefront's step stand behind the
// wait for the second half's weights, which has nothing beside it. That wait counts
// the row loads of step t + 2 as well, which went out just before, so their latency
// lies open in every step and the third stage hides nothing; and both halves'
// operands are live together (246 registers at 128 rows, 160 at 64).
//
// Measured on MI355X, 256 experts of 7168 -> 2 x 2048: 32768 tokens x 8 rows 4.38 ms
// (15.4 TFLOP, 3.5 PFLOP/s; the matrix cores busy 45 % at a clock held near 1.9 GHz),
// 4096 tokens x 8 skewed 0.97 ms (4.25 GB, 4.4 TB/s). A version of the former that took
// 4.5 ms took 3.2 without its loads, 3.6 without the weights', 4.0 without the rows',
// 4.1 without the exchange of dwords: what those cost beside these waits.
constexpr int kWaves = 4;               // along the features
constexpr int kStages = 3;              // 256-element steps of rows in LDS
constexpr int kBand = 8;
constexpr int kChunkGroups = 240;       // groups of 32 whose scales LDS holds
constexpr int kRowWords = kChunkGroups / 4;

template <bool GATED, int ROWS>
__global__ __launch_bounds__(kWaves * 64, 2)
void expert_mx4_kernel(const char* __restrict__ rows, const uint8_t* __restrict__ row_scales,
                       const char* __restrict__ w, const uint8_t* __restrict__ scales,
                       const int32_t* __restrict__ offsets, int32_t E, int32_t max_rows,
                       int32_t red, int32_t feats, int32_t ftiles, int32_t act,
                       char* __restrict__ out, int32_t zero, int32_t chunk) {
    // Output features of a wavefront: half its blocks are up rows if gated.
    constexpr int kFeats = kBlocks * 16 / (GATED ? 2 : 1);
    typedef PackedOperand<ROWS, kWaves> Rows;
    __shared__ v4i lds[kStages * Rows::kChunks];
    __shared__ uint32_t scale_lds[ROWS * kChunkGroups / 4];
    __shared__ int32_t info[4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t number = expert_tile_number(chunk);
    if (wave == 0) {
        const ExpertTile t = expert_find_tile(offsets, E, max_rows, ROWS, ftiles, kBand, number);
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
    const int32_t steps = (red + 255) / 256;
    const int32_t halves = (red + kMxfp4Step - 1) / kMxfp4Step;
    const int32_t groups = red / 32;

    // This wavefront's blocks; those past the matrix read its last one and are
    // not stored.
    const int32_t nb = (feats + 15) / 16;
    auto block_of = [&](int b) {
        const bool up = GATED && b >= kBlocks / 2;
        const int32_t ob = min(f0 / 16 + (GATED ? b % (kBlocks / 2) : b), nb - 1);
        return (int64_t(e) * (GATED ? 2 : 1) + (up ? 1 : 0)) * nb + ob;
    };
    const char* wb[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) wb[b] = w + block_of(b) * halves * 1024;
    // Lane group g loads the scales of block g.
    const uint8_t* sb = scales + block_of(g) * halves * 64 + i * 4;

    // The rows' scales of kChunkGroups groups from c0 on to LDS. Of row r, word 15
    // g + q holds scale group g of the four half steps from 4 q on, a byte each: what
    // lane group g needs for two steps, one of whose bytes a product picks by
    // itself. 60 words a row and 15 a group put the 64 lanes into as many banks.
    // Groups behind the sum's end get 1: they meet weights of zero.
    const uint8_t* sbase = row_scales + int64_t(row0) * groups;
    auto load_scales = [&](int32_t c0) {
        const int32_t len = min(groups - c0, kChunkGroups);
        const int32_t quads = (len + 15) / 16;
        for (int q = threadIdx.x; q < nrows * quads; q += kWaves * 64) {
            const int r = q / quads, at = q % quads * 16;
            const uint8_t* p = sbase + r * groups + c0 + at;
            v4i v;
            if (at + 16 <= len) {
                __builtin_memcpy(&v, p, 16);
            } else {
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const uint32_t byte = at + k < len ? p[k] : 127;
                    const uint32_t word = k % 4 == 0 ? 0 : static_cast<uint32_t>(v[k / 4]);
                    v[k / 4] = static_cast<int32_t>(word | byte << (8 * (k % 4)));
                }
            }
            const uint32_t a = __builtin_amdgcn_perm(v[1], v[0], 0x05010400u);
            const uint32_t b = __builtin_amdgcn_perm(v[3], v[2], 0x05010400u);
            const uint32_t c = __builtin_amdgcn_perm(v[1], v[0], 0x07030602u);
            const uint32_t d = __builtin_amdgcn_perm(v[3], v[2], 0x07030602u);
            uint32_t* to = scale_lds + r * kRowWords + at / 16;
            to[0] = __builtin_amdgcn_perm(b, a, 0x05040100u);
            to[kRowWords / 4] = __builtin_amdgcn_perm(b, a, 0x07060302u);
            to[kRowWords / 2] = __builtin_amdgcn_perm(d, c, 0x05040100u);
            to[kRowWords / 4 * 3] = __builtin_amdgcn_perm(d, c, 0x07060302u);
        }
    };

    auto run = [&](auto row_blocks) {
        constexpr int NB = decltype(row_blocks)::value;
        Rows rt;
        const int64_t pitch = red / 2;
        const char* rbase = rows + int64_t(row0) * pitch;
        rt.init(wave, lane, 0, pitch, [&](int) { return rbase; },
                [&](int p) { return min(p, nrows - 1); });
        f32x4 acc[kBlocks][NB];
#pragma unroll
        for (int a = 0; a < kBlocks; ++a)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        // What a half step of 128 elements takes from memory to registers.
        struct Half {
            v4i q[kBlocks];
            uint32_t scale;
        };
        auto issue_rows = [&](int32_t t, int stage) {
            v4i* buf = lds + stage * Rows::kChunks;
            const int left = min(red / 4 - t * 64, 64);         // in pairs of bytes
            if (left == 64)
                rt.issue(t, buf);
            else
                rt.issue_partial(t, left, lane, buf);
        };
        auto load = [&](int32_t half, Half& d) {
            // A uniform address and a 32-bit offset per lane.
            uint32_t qo = lane * 16;
            reform(qo);
            const int32_t at = min(half, halves - 1);
            d.scale = *reinterpret_cast<const uint32_t*>(sb + int64_t(at) * 64);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
                d.q[b] = *reinterpret_cast<const v4i*>(wb[b] + int64_t(at) * 1024 + qo);
        };
        const int shift = 8 * g;
        auto order = [&](Half& d, uint32_t (&sc)[kBlocks]) {
            spread(d.scale, sc);
#pragma unroll
            for (int a = 0; a < kBlocks; ++a) {
                sc[a] >>= shift;
                d.q[a] = by_groups(d.q[a]);
            }
        };
        // Two row blocks' operands, read while the products of the two before them
        // run.
        constexpr int kPair = NB == 1 ? 1 : 2;
        struct Pair {
            v4i x[kPair];
        };
        auto fetch = [&](Pair& d, const v4i* buf, int b, int h) {
#pragma unroll
            for (int k = 0; k < kPair; ++k)
                if (b + k < NB) d.x[k] = __builtin_bit_cast(v4i, rt.frag(buf, b + k, h));
        };
        int32_t rs[NB];                         // the rows' scales of four half steps
        auto multiply = [&](const Half& d, const uint32_t (&sc)[kBlocks], const v4i* buf,
                            auto half) {
            constexpr int kHalf = decltype(half)::value;        // of four
            Pair p[2];
            fetch(p[0], buf, 0, kHalf & 1);
#pragma unroll
            for (int b = 0; b < NB; b += kPair) {
                if (b + kPair < NB) fetch(p[b / kPair % 2 ^ 1], buf, b + kPair, kHalf & 1);
                __builtin_amdgcn_sched_barrier(0);
                const Pair& now = p[b / kPair % 2];
#pragma unroll
                for (int k = 0; k < kPair; ++k)
#pragma unroll
                    for (int a = 0; a < kBlocks; ++a)
                        if (b + k < NB)
                            acc[a][b + k] = multiply4<kHalf>(d.q[a], sc[a], now.x[k], rs[b + k],
                                                             acc[a][b + k]);
            }
        };

        Half lo, hi;
        uint32_t sc[kBlocks];
        issue_rows(0, 0);
        if (steps > 1) issue_rows(1, 1);
        load(0, lo);
        load(1, hi);
        load_scales(0);
        wait_loads<0>();
        step_barrier();
        int stage = 0;
        auto step = [&](auto odd, int32_t t) {
            constexpr int kOdd = decltype(odd)::value;
            const int after = stage + 1 == kStages ? 0 : stage + 1;
            const int free = after + 1 == kStages ? 0 : after + 1;
            const v4i* buf = lds + stage * Rows::kChunks;
            order(lo, sc);
            __builtin_amdgcn_sched_barrier(0);
            // Behind the first use of this step's registers: the wait for the first
            // half does not wait for these loads. The one for the second half does.
            if (t + 2 < steps) issue_rows(t + 2, free);
            multiply(lo, sc, buf, std::integral_constant<int, 2 * kOdd>{});
            __builtin_amdgcn_sched_barrier(0);
            load(2 * t + 2, lo);
            __builtin_amdgcn_sched_barrier(0);
            order(hi, sc);
            if (2 * t + 1 >= halves) {
                // A sum that ends in the first half. The first half's products are
                // placed behind this branch.
#pragma unroll
                for (int a = 0; a < kBlocks; ++a) hi.q[a] = v4i{0, 0, 0, 0};
            }
            multiply(hi, sc, buf, std::integral_constant<int, 2 * kOdd + 1>{});
            __builtin_amdgcn_sched_barrier(0);
            load(2 * t + 3, hi);
            __builtin_amdgcn_sched_barrier(0);
            // The next step's rows have landed: this step's registers, which
            // were waited for, were loaded behind them.
            step_barrier();
            stage = after;
        };
        int32_t first = 0;                      // group the scales in LDS begin with
        for (int32_t t = 0; t < steps; t += 2) {
            if (8 * t - first == kChunkGroups) {
                // Every wavefront is past the last barrier: the old ones are read.
                first = 8 * t;
                load_scales(first);
                __syncthreads();
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)        // rows past the last are not stored
                rs[b] = static_cast<int32_t>(
                    scale_lds[(b * 16 + i) * kRowWords + g * (kRowWords / 4) + (8 * t - first) / 16]);
            step(std::integral_constant<int, 0>{}, t);
            if (t + 1 < steps) step(std::integral_constant<int, 1>{}, t + 1);
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
                    for (int k = 0; k < 4; ++k)
                        v[k] = activate(act, acc[a][b][k]) * acc[a + 2][b][k];
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
    else if (nrows <= 48 || ROWS == 64) {
        if (nrows <= 48)
            run(std::integral_constant<int, 3>{});
        else
            run(std::integral_constant<int, 4>{});
    } else if constexpr (ROWS == 128) {
        if (nrows <= 64)
            run(std::integral_constant<int, 4>{});
        else if (nrows <= 96)
            run(std::integral_constant<int, 6>{});
        else
            run(std::integral_constant<int, 8>{});
    }
}

// ---- Few rows per expert --------------------------------------------------
//
// As the streamed products with bf16 rows: 64 features and up to 16 rows per
// workgroup, the sum split over its wavefronts and joined in LDS in wavefront
// order. Rows are small enough to come straight from the caches. Bound: the weights'
// bytes, but for the start and end of a launch; one token's 8 experts of 7168 -> 2 x
// 2048 take 19.8 us on MI355X (125 MB, 6.3 TB/s; passes over the same state find part
// of them in the memory-side cache).
constexpr int kStreamWaves = 4;
constexpr int kStreamRows = 16;
constexpr int kStreamChunk = 32;

template <bool GATED>
__global__ __launch_bounds__(kStreamWaves * 64, 4)
void expert_mx4_stream_kernel(const char* __restrict__ rows, const uint8_t* __restrict__ row_scales,
                              const char* __restrict__ w, const uint8_t* __restrict__ scales,
                              const int32_t* __restrict__ offsets, int32_t E, int32_t max_rows,
                              int32_t red, int32_t feats, int32_t ftiles, int32_t act,
                              char* __restrict__ out, int32_t zero, int32_t chunk) {
    constexpr int kFeatBlocks = GATED ? kBlocks / 2 : kBlocks;  // of the output
    __shared__ f32x4 part[kStreamWaves][kBlocks][64];
    __shared__ int32_t info[4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t number = expert_tile_number(chunk);
    if (wave == 0) {
        const ExpertTile t = expert_find_tile(offsets, E, max_rows, kStreamRows, ftiles, 4, number);
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
    const int32_t steps = (red + kMxfp4Step - 1) / kMxfp4Step;
    const int32_t groups = red / 32;
    auto block_of = [&](int b) {
        const int32_t nb = (feats + 15) / 16;
        const bool up = GATED && b >= kFeatBlocks;
        return int64_t(e) * nb * (GATED ? 2 : 1) + (up ? nb : 0) +
               min(f0 / 16 + (GATED ? b % kFeatBlocks : b), nb - 1);
    };
    const char* wb[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) wb[b] = w + block_of(b) * steps * 1024;
    const uint8_t* sb = scales + block_of(g) * steps * 64 + i * 4;
    const int64_t row = row0 + min(i, nrows - 1);
    const char* rbase = rows + row * (red / 2);
    const uint8_t* sbase = row_scales + row * groups;

    struct Step {
        v4i q[kBlocks];
        uint32_t scale;
        v4i x;
        int32_t rs;
    };
    auto load = [&](int32_t t, Step& d) {
        const int32_t group = min(4 * t + g, groups - 1);
        uint32_t qo = lane * 16;
        reform(qo);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
            d.q[b] = __builtin_nontemporal_load(
                reinterpret_cast<const v4i*>(wb[b] + int64_t(t) * 1024 + qo));
        d.scale = *reinterpret_cast<const uint32_t*>(sb + int64_t(t) * 64);
        d.x = *reinterpret_cast<const v4i*>(rbase + int64_t(group) * 16);
        d.rs = sbase[group];
        __builtin_amdgcn_sched_barrier(0);
    };
    f32x4 acc[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto compute = [&](const Step& d) {
        uint32_t sc[kBlocks];
        spread(d.scale, sc);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
            acc[b] = multiply4<0>(by_groups(d.q[b]), sc[b] >> (8 * g), d.x, d.rs, acc[b]);
    };
    // Wavefront w takes steps w, w + kStreamWaves, ..., two in flight.
    Step even, odd;
    int32_t t = wave;
    if (t < steps) load(t, even);
    if (t + kStreamWaves < steps) load(t + kStreamWaves, odd);
    while (t < steps) {
        compute(even);
        if (t + 2 * kStreamWaves < steps) load(t + 2 * kStreamWaves, even);
        t += kStreamWaves;
        if (t >= steps) break;
        compute(odd);
        if (t + 2 * kStreamWaves < steps) load(t + 2 * kStreamWaves, odd);
        t += kStreamWaves;
    }

#pragma unroll
    for (int b = 0; b < kBlocks; ++b) part[wave][b][lane] = acc[b];
    __syncthreads();
    if (wave >= kFeatBlocks) return;
    f32x4 v = part[0][wave][lane];
#pragma unroll
    for (int p = 1; p < kStreamWaves; ++p) v += part[p][wave][lane];
    if constexpr (GATED) {
        f32x4 u = part[0][wave + kFeatBlocks][lane];
#pragma unroll
        for (int p = 1; p < kStreamWaves; ++p) u += part[p][wave + kFeatBlocks][lane];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = activate(act, v[k]) * u[k];
    }
    const int32_t f = f0 + wave * 16 + g * 4;
    if (i >= nrows || f >= feats) return;
    *reinterpret_cast<v2i*>(out + (int64_t(row0 + i) * feats + f) * 2) = pack_bf16x4(v);
}

int64_t tile_features(bool gated, int32_t feats) {
    const int32_t per = kWaves * kBlocks * 16 / (gated ? 2 : 1);
    return (int64_t(feats) + per - 1) / per;
}
int64_t tiles_of(bool gated, int32_t E, int64_t max_rows, int32_t feats, int rows) {
    return tile_features(gated, feats) *
           ((max_rows + rows - 1) / rows + (max_rows < E ? max_rows : E));
}
int tile_rows(const ExpertMx4Args& a) {
    return expert_mx4_tile_rows(a.gated, a.E, a.max_rows, a.feats);
}
int64_t tiles_of(const ExpertMx4Args& a) {
    return tiles_of(a.gated, a.E, a.max_rows, a.feats, tile_rows(a));
}
int64_t round_up(int64_t n, int64_t unit) { return (n + unit - 1) / unit * unit; }
int64_t active(const ExpertMx4Args& a) { return a.max_rows < a.E ? a.max_rows : a.E; }

// Neighbouring tiles that one XCD takes together: with 64 an expert's rows are
// read into few L2 caches (256 experts of 7168 -> 2 x 2048 at 1024 rows each 4.49
// ms, with 8 4.65; 64 rows each 0.72 with both). Fewer where that would leave an
// XCD fewer than 8 such pieces.
int32_t tile_chunk(const ExpertMx4Args& a) {
    const int64_t tiles = tiles_of(a);
    int32_t chunk = 1;
    while (chunk < 64 && tiles >= int64_t(chunk) * 2 * kExpertXcds * 8) chunk *= 2;
    return chunk;
}
int64_t tile_workgroups(const ExpertMx4Args& a) {
    return round_up(tiles_of(a), int64_t(kExpertXcds) * tile_chunk(a));
}
int64_t stream_features(const ExpertMx4Args& a) {
    const int32_t per = (a.gated ? kBlocks / 2 : kBlocks) * 16;
    return (int64_t(a.feats) + per - 1) / per;
}
int64_t stream_workgroups(const ExpertMx4Args& a) {
    return round_up(stream_features(a) * ((a.max_rows + kStreamRows - 1) / kStreamRows + active(a)),
                    int64_t(kExpertXcds) * kStreamChunk);
}

template <class Kernel>
hipError_t launch(Kernel kernel, int64_t workgroups, int threads, int64_t ftiles, int32_t chunk,
                  const ExpertMx4Args& a, hipStream_t stream) {
    const char* w = static_cast<const char*>(a.w);
    const char* scales = w + mxfp4_tiles(a.E, a.gated ? 2 * a.feats : a.feats, a.red) * 1024;
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(workgroups)), dim3(threads), 0, stream,
                       static_cast<const char*>(a.rows), static_cast<const uint8_t*>(a.row_scales),
                       w, reinterpret_cast<const uint8_t*>(scales), a.offsets, a.E,
                       static_cast<int32_t>(a.max_rows), a.red, a.feats,
                       static_cast<int32_t>(ftiles), a.activation, static_cast<char*>(a.out),
                       a.zero, chunk);
    return hipGetLastError();
}

}  // namespace

// Measured on MI355X, 64 against 128 rows per tile, other weights in every call: 64
// experts of 7168 -> 2 x 2048 at 32 rows each 176 and 177 us, at 64 212 and 183, at
// 256 398 and 354; 8 of 4096 -> 2 x 1408 at 128 24.1 and 29.8 (176 tiles of 128
// rows), at 256 30.8 and 30.9 (264), at 512 42.8 and 41.8 (440); 24 of 1984 -> 1000
// at 256 21.4 and 21.9 (288), at 512 37.7 and 31.7 (480).
int expert_mx4_tile_rows(bool gated, int32_t E, int64_t max_rows, int32_t feats) {
    return max_rows >= 64 * int64_t(E) && tiles_of(gated, E, max_rows, feats, 128) >= 320 ? 128
                                                                                          : 64;
}

int64_t expert_mx4_grid(const ExpertMx4Args& a) { return tile_workgroups(a) * (kWaves * 64); }
int64_t expert_mx4_stream_grid(const ExpertMx4Args& a) {
    return stream_workgroups(a) * (kStreamWaves * 64);
}

hipError_t launch_expert_mx4(const ExpertMx4Args& a, hipStream_t stream) {
    auto kernel = tile_rows(a) == 128
                      ? (a.gated ? expert_mx4_kernel<true, 128> : expert_mx4_kernel<false, 128>)
                      : (a.gated ? expert_mx4_kernel<true, 64> : expert_mx4_kernel<false, 64>);
    return launch(kernel, tile_workgroups(a), kWaves * 64, tile_features(a.gated, a.feats),
                  tile_chunk(a), a, stream);
}

hipError_t launch_expert_mx4_stream(const ExpertMx4Args& a, hipStream_t stream) {
    return launch(a.gated ? expert_mx4_stream_kernel<true> : expert_mx4_stream_kernel<false>,
                  stream_workgroups(a), kStreamWaves * 64, stream_features(a), kStreamChunk, a,
                  stream);
}

}  // namespace moe
